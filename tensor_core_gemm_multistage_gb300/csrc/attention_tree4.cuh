// attention_tree4.cuh - attention of drafted tokens over a paged cache of 4 bits (one token a request is
// ordinary decoding).
//
// A key (value) is s code + m for each 64 of its dimensions, so with the codes c and C of a key and a value
//   score_j = sum_g s_jg (q_g . c_jg) + m_jg sum(q_g),
//   O = sum_j p_j s_jg (C_jg - 8) + sum_j p_j (m_jg + 8 s_jg):
// both products run on the codes themselves, and scales and minima are applied to their results and to p, in fp32.
// A code is an fp16 operand as it lies: 4 bits low in a half are the subnormal c 2^-24, the next 4 bits c 2^-20,
// which tensor cores multiply exactly; the powers of two go into the queries, and off the sums at the end.  So
// unpacking takes one AND for two values, and a shift for four.  The 8 (which halves what rounding p s to 16 bits
// does to O) leaves chunk by chunk with the sum of the rounded p s, a product with ones: left to the end it would cost
// digits (4096 keys, fp16: 3.1e-4 of O), and as products with the constant -8 it took 10 us more of 161 (16
// trees of 40 nodes over 4096 tokens, 8 heads of 4 queries each).  Queries are held
// as fp16 times a power of two for each row (bf16's 8 bits fit; what is 2^-25 of the row's largest loses digits; from
// 2^112 on, where the power of two that undoes it would overflow, a row is NaN).
//
// What bounds it: D / 2 + D / 16 bytes a key and head, twice, from HBM; per byte that is 3.6 times the
// arithmetic of a 16-bit cache, so the instructions that unpack codes come next.  Codes are therefore unpacked
// in registers into mma.sync operands: operands of tcgen05 come from shared memory or TMEM, and the unpacked rows
// would be written there and read again, 93 of an SM's 128 bytes a clock at HBM's rate, before the first product.
// Where many rows share a key that would be no hindrance; but 128 rows on tcgen05, two CTAs an SM, took 175 us for 16
// trees of 40 nodes: product, scores, p s and product follow one another, 6500 clocks for 64 keys.  Measured, D = 128, 8
// heads of keys, 32 of queries: 48 requests of 4000 to 8000 tokens 75 us (4.3 TB/s), 16 trees of 40 nodes over up to 4096
// tokens 155 us (148 TFLOP/s; a warp's own latencies, with two warps a scheduler). The 75 us are no unit's limit either: issue 57 %,
// integer pipe 48 %, tensor cores 25 %, with four CTAs of 128 registers an SM.
// Keys are the products' rows (16 at once) and the rows of queries that share them, nodes x group, their columns (8): no row
// is padding whatever the group, and no column where nodes x group is a multiple of 8.  With one token and 4 queries a key
// head half of the columns are padding, and of the lanes that compute scores and probabilities after them.
//
// Split.  A CTA's four warps take 32-key chunks of one request, head and tile of 8 NT query rows in turn; each warp
// copies its own chunks (cp.async) and has its own softmax state, and the states are joined in shared memory.
//  * Little work: a cluster of CTAs shares an item's chunks and joins their states by distributed shared
//    memory.  One launch, no workspace.
//  * Much: the chunks of all items are laid end to end and shared out evenly over as many CTAs as the SMs hold at
//    once, whatever the lengths (each CTA finds its range by one sum over the requests).  An item that one CTA covers
//    is written at once, else its CTAs leave their states in the workspace, two a CTA at most, and a second
//    launch joins them in the CTAs' order.  (Clusters there cost a start and a join a wave, and waves leave SMs idle: 84 us
//    for 79, 48 requests.)
// No order changes from run to run.
#pragma once

#include <atomic>
#include <climits>
#include <type_traits>

#include "gsr.h"
#include "ptx_attention.cuh"
#include "rows16.cuh"
#include "serving.h"

namespace gsr {
namespace {

constexpr int kT4Threads = 32 * kT4Warps;

struct Tree4Plan {
    Divider by_page;
    int tiles;                  // tiles of query rows a request and head
    int cluster;                // CTAs that share an item; 0: shared out evenly
    int chunks;                 // that a table's row can hold
};

// What a request has: query rows (nodes x group) from q0 on, cached tokens `kv`, of them `ctx` before the tree,
// `n` in the table; units of work: chunks (one at least) of each of its items.
struct T4Request {
    int q0, rows, nodes, ctx, n, chunks, tiles;
    __device__ __forceinline__ long long units(int heads) const { return (long long)heads * tiles * max(chunks, 1); }
};
template <int ROWS>
__device__ __forceinline__ T4Request t4_request(const Tree4Params& p, int b) {
    const int q0 = __ldg(p.q_starts + b), q1 = __ldg(p.q_starts + b + 1), kv = __ldg(p.kv_lens + b);
    T4Request r;
    r.q0 = q0;
    r.nodes = q0 < 0 ? 0 : max(min(min(q1 - q0, p.max_nodes), p.total_q - q0), 0);
    r.rows = r.nodes * p.group;
    r.tiles = (r.rows + ROWS - 1) / ROWS;
    r.ctx = kv - (q1 - q0);
    r.n = (int)min((long long)kv, (long long)p.table_width * p.page);
    r.chunks = r.n > 0 ? (r.n + kT4Keys - 1) / kT4Keys : 0;
    return r;
}

template <class Type, int Dim, int Nt>
struct T4Cfg {
    using T = Type;
    static constexpr int D = Dim, NT = Nt, G = D / 64, ROWS = 8 * NT;
    static constexpr int STAGES = NT == 1 ? 2 : 3, CTAS = Tree4Split::ctas_an_sm(NT, Dim);
    static constexpr int CODES = D / 2, PARAMS = D / 16;             // bytes of a row
    static constexpr int STAGE = kT4Keys * 2 * (CODES + PARAMS);
    static constexpr int RING = kT4Warps * STAGES * STAGE;
    static constexpr int FACTORS = kT4Keys * (D == 128 ? 40 : 24);   // bytes of a warp's chunk: see key_factors
    static constexpr int SMEM = RING + kT4Warps * FACTORS;
    static constexpr int PITCH = D + 2;                              // floats of a row's state: M, l, D sums
    static constexpr int PART = ROWS * PITCH;                        // floats of a warp's states
    static_assert((kT4Warps + 1) * PART * 4 <= RING, "states are joined in the ring");
};

__device__ __forceinline__ uint32_t t4_smem(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool real) {       // zeros where not real
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(real ? BYTES : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float lg2_fast(float x) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Codes 0 and 4 of a word as two operands, c 2^-24; codes 1 and 5, c 2^-20.
__device__ __forceinline__ uint32_t codes_low(uint32_t w) { return w & 0x000f000fu; }
__device__ __forceinline__ uint32_t codes_high(uint32_t w) { return w & 0x00f000f0u; }
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float4 lds128(uint32_t a) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ void sts128(uint32_t a, float x, float y, float z, float w) {
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(x), "f"(y), "f"(z), "f"(w) : "memory");
}
__device__ __forceinline__ void sts64(uint32_t a, float x, float y) {
    asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(x), "f"(y) : "memory");
}
// Two 16 x 16 blocks of bytes, transposed: rows of 16 bytes at the addresses of lanes 0 to 15 and 16 to 31.  Lane 4 g + t
// gets column g of rows 4 t to 4 t + 3 in v[0], column g + 8 in v[1], the second block's in v[2] and v[3].
__device__ __forceinline__ void load_transposed(uint32_t (&v)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(a)
                 : "memory");
}

// Where 16-byte piece c of key k's codes lies in a stage: neither the eight keys that a transposed load reads at once nor
// the four keys 2 apart that a product's rows are read from meet in a bank.
template <int D>
__device__ __forceinline__ int code_at(int k, int c) {
    if constexpr (D == 128) return ((k & ~3) | (k & 1) << 1 | (k >> 1 & 1)) * 64 + (c ^ ((k >> 2 & 1) << 1 | (k & 1))) * 16;
    return ((k & 16) | (k & 1) << 3 | (k >> 1 & 7)) * 32 + (c ^ (k & 1)) * 16;
}
// Keys in the order in which products have them as rows: the even ones of 16, then the odd ones.
__device__ __forceinline__ int row_of(int k) { return (k & 16) | (k & 1) << 3 | (k >> 1 & 7); }

// A chunk's keys as the arithmetic takes them, each prepared by one lane, since four lanes of the products need each:
// of K scales and minima; of V, with s the largest of the key's scales, their ratios to it, (m + 8 s') / s, log2 s, 1 / s.
// With p s' = 2^(score + log2 s - base) (s' / s), what is rounded to fp16 for the second product stays in range
// whatever the values' size.
template <class T, int D>
__device__ __forceinline__ void key_factors(uint32_t params_k, uint32_t params_v, uint32_t to, int lane) {
    const int row = row_of(lane);
    auto largest = [](float s) { return fminf(fmaxf(s, 0x1p-24f), 0x1p124f); };
    if constexpr (D == 128) {
        const uint2 k = lds64(params_k + 8 * lane), v = lds64(params_v + 8 * lane);
        const float2 k0 = Pair<T>::unpack(k.x), k1 = Pair<T>::unpack(k.y), v0 = Pair<T>::unpack(v.x), v1 = Pair<T>::unpack(v.y);
        const float s = largest(fmaxf(v0.x, v1.x)), inv = rcp_fast(s), r0 = v0.x * inv, r1 = v1.x * inv;
        sts128(to + 16 * row, k0.x, k1.x, k0.y, k1.y);
        sts128(to + 512 + 16 * row, r0, r1, fmaf(8.0f, r0, v0.y * inv), fmaf(8.0f, r1, v1.y * inv));
        sts64(to + 1024 + 8 * row, lg2_fast(s), inv);
    } else {
        const float2 k = Pair<T>::unpack(lds32(params_k + 4 * lane)), v = Pair<T>::unpack(lds32(params_v + 4 * lane));
        const float s = largest(v.x), inv = rcp_fast(s), r = v.x * inv;
        sts64(to + 8 * row, k.x, k.y);
        sts128(to + 256 + 16 * row, r, fmaf(8.0f, r, v.y * inv), lg2_fast(s), inv);
    }
    __syncwarp();
}
template <int D, int G>
__device__ __forceinline__ void factors_k(uint32_t at, int row, float (&s)[G], float (&m)[G]) {
    if constexpr (D == 128) {
        const float4 x = lds128(at + 16 * row);
        s[0] = x.x;
        s[1] = x.y;
        m[0] = x.z;
        m[1] = x.w;
    } else {
        const uint2 x = lds64(at + 8 * row);
        s[0] = __uint_as_float(x.x);
        m[0] = __uint_as_float(x.y);
    }
}
template <int D, int G>
__device__ __forceinline__ void factors_v(uint32_t at, int row, float (&ratio)[G], float (&centre)[G], float& log_s, float& inv) {
    if constexpr (D == 128) {
        const float4 x = lds128(at + 512 + 16 * row);
        const uint2 y = lds64(at + 1024 + 8 * row);
        ratio[0] = x.x;
        ratio[1] = x.y;
        centre[0] = x.z;
        centre[1] = x.w;
        log_s = __uint_as_float(y.x);
        inv = __uint_as_float(y.y);
    } else {
        const float4 x = lds128(at + 256 + 16 * row);
        ratio[0] = x.x;
        centre[0] = x.y;
        log_s = x.z;
        inv = x.w;
    }
}

// States of row q from `count` places, each state_of(i, place): largest M, and sums weighed by 2^(M_i - M).
template <class C, class State>
__device__ __forceinline__ void t4_join(State state_of, int count, int q, int d, float& most, float& sum, float2& v) {
    most = -INFINITY;
    for (int i = 0; i < count; ++i) most = fmaxf(most, state_of(i, q * C::PITCH));
    sum = 0.0f;
    v = make_float2(0.0f, 0.0f);
    if (most == -INFINITY) return;
    for (int i = 0; i < count; ++i) {
        const float mi = state_of(i, q * C::PITCH);
        if (mi == -INFINITY) continue;                 // that part saw nothing; its sums are not written
        const float f = exp2_fast(mi - most);
        sum = fmaf(f, state_of(i, q * C::PITCH + 1), sum);
        v.x = fmaf(f, state_of(i, q * C::PITCH + 2 + d), v.x);
        v.y = fmaf(f, state_of(i, q * C::PITCH + 3 + d), v.y);
    }
}

struct T4Shared {
    uint64_t sees[GSR_TREE_MAX_NODES];       // bit u of sees[t]: node t sees node u
    int parent[GSR_TREE_MAX_NODES];
};

// Chunks first + i step (of this warp) below `end` of an item; false where the tile has no rows.  out(write, q, d, most,
// sum, v): the CTA's joined state of row q, dimensions d and d + 1 (write(q, d, x, y, sum) puts them into O).
template <class C, class Out>
__device__ __forceinline__ bool t4_part(const Tree4Params& p, const Tree4Plan& plan, char* smem, T4Shared& sh, int b, int h, int tile, int first,
                                        int step, int end, Out out) {
    using T = typename C::T;
    constexpr int D = C::D, G = C::G, NT = C::NT;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int* table = p.table + (long long)b * p.table_width;

    // ---- the pages of a chunk: eight keys lie in one; a lane looks after keys 8 (lane / 8) on
    const int part = lane >> 3, j8 = lane & 7;
    auto look_up = [&](int chunk) {                         // whatever the length is: entries of the table are there
        const int col = plan.by_page(min(chunk, plan.chunks) * kT4Keys + 8 * part);
        return col < p.table_width ? __ldg(table + col) : -1;
    };
    int pages[C::STAGES + 1];                               // of the chunks in flight, and of the next two
#pragma unroll
    for (int i = 0; i <= C::STAGES; ++i) pages[i] = look_up(first + i * step);

    const T4Request req = t4_request<C::ROWS>(p, b);
    const int q0 = req.q0, nodes = req.nodes, rows = req.rows, ctx = req.ctx, n = req.n, chunks = min(req.chunks, end);
    if (tile * C::ROWS >= rows) return false;

    // ---- the copies of a chunk
    constexpr int PIECES = C::CODES / 16, AT_ONCE = 8 / PIECES;             // 16-byte pieces of a row, rows of eight lanes
    const uint32_t ring = t4_smem(smem) + warp * C::STAGES * C::STAGE;
    const char* const k_codes = p.K.codes.data + (long long)(j8 / PIECES) * p.K.codes.row + h * p.K.codes.head + 16 * (j8 % PIECES);
    const char* const v_codes = p.V.codes.data + (long long)(j8 / PIECES) * p.V.codes.row + h * p.V.codes.head + 16 * (j8 % PIECES);
    const char* const k_params = p.K.params.data + j8 * p.K.params.row + h * p.K.params.head;
    const char* const v_params = p.V.params.data + j8 * p.V.params.row + h * p.V.params.head;
    auto at_row = [](const char* base, const Bytes& t, uint32_t page, uint32_t row) {      // strides are below 2^32
        return base + (unsigned long long)page * (uint32_t)t.page + (unsigned long long)row * (uint32_t)t.row;
    };
    auto there_is = [&](int page) { return page >= 0 && page < p.num_pages; };
    auto copy = [&](int chunk, int stage, int pg) {
        const uint32_t at = ring + stage * C::STAGE;
        const int key = chunk * kT4Keys + 8 * part, real = there_is(pg) ? n - key : 0;    // of these eight keys, those that are there
        const uint32_t page = there_is(pg) ? pg : 0, row = key - plan.by_page(key) * p.page;   // the others' addresses are a page's all the same
        const char *k = at_row(k_codes, p.K.codes, page, row), *v = at_row(v_codes, p.V.codes, page, row);
        const uint32_t params = at + 2 * kT4Keys * C::CODES + lane * C::PARAMS;
        const char *pk = at_row(k_params, p.K.params, page, row), *pv = at_row(v_params, p.V.params, page, row);
        if (__all_sync(0xffffffffu, real >= 8)) {
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
                const uint32_t to = at + code_at<D>(8 * part + j8 / PIECES + i * AT_ONCE, j8 % PIECES);
                copy_async<16>(to, k + i * AT_ONCE * p.K.codes.row, true);
                copy_async<16>(to + kT4Keys * C::CODES, v + i * AT_ONCE * p.V.codes.row, true);
            }
            copy_async<C::PARAMS>(params, pk, true);
            copy_async<C::PARAMS>(params + kT4Keys * C::PARAMS, pv, true);
            return;
        }
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int r = j8 / PIECES + i * AT_ONCE;
            const uint32_t to = at + code_at<D>(8 * part + r, j8 % PIECES);
            copy_async<16>(to, k + i * AT_ONCE * p.K.codes.row, r < real);
            copy_async<16>(to + kT4Keys * C::CODES, v + i * AT_ONCE * p.V.codes.row, r < real);
        }
        copy_async<C::PARAMS>(params, pk, j8 < real);
        copy_async<C::PARAMS>(params + kT4Keys * C::PARAMS, pv, j8 < real);
    };
#pragma unroll
    for (int i = 0; i < C::STAGES - 1; ++i) {
        if (first + i * step < chunks) copy(first + i * step, i, pages[i]);
        copies_commit();
    }

    // ---- which nodes see which
    if (threadIdx.x < nodes) sh.parent[threadIdx.x] = p.parents ? __ldg(p.parents + q0 + threadIdx.x) : (int)threadIdx.x - 1;
    __syncthreads();
    if (threadIdx.x < nodes) {
        int u = threadIdx.x;
        uint64_t bits = 1ull << u;
        if (!p.parents) bits = bits * 2 - 1;
        else
            for (int up = sh.parent[u]; up >= 0 && up < u; up = sh.parent[u]) {
                bits |= 1ull << up;
                u = up;
            }
        sh.sees[threadIdx.x] = bits;
    }

    // ---- queries: the products' second operand, columns n of 8, their sums of each 64 dimensions, and the factor of scores
    uint32_t qf[G][2][2][NT][2];
    float qsum[G][NT][2], factor[NT][2];
    const float plain = p.score.cap_out != 0.0f ? p.score.cap_in : p.score.sl2;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = tile * C::ROWS + 8 * nt + g, node = r / p.group;
        const T* q = static_cast<const T*>(p.Q) + (q0 + node) * p.q_row + (h * p.group + r % p.group) * p.q_head;
        uint4 raw[G][2];
#pragma unroll
        for (int gi = 0; gi < G; ++gi)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                raw[gi][w] = make_uint4(0u, 0u, 0u, 0u);
                if (r < rows) raw[gi][w] = *reinterpret_cast<const uint4*>(q + 64 * gi + 16 * t + 8 * w);
            }
        uint32_t largest = 0u;                             // bits of the largest |q|
#pragma unroll
        for (int gi = 0; gi < G; ++gi)
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = Pair<T>::unpack((&raw[gi][w].x)[i]);
                    largest = max(largest, max(__float_as_uint(fabsf(f.x)), __float_as_uint(fabsf(f.y))));
                }
        largest = max(largest, __shfl_xor_sync(0xffffffffu, largest, 1));
        largest = max(largest, __shfl_xor_sync(0xffffffffu, largest, 2));
        // the row times 2^e is below 2^11 beside c 2^-20, and 16 times that beside c 2^-24; 16 2^e and 2^-e 2^20 are floats
        const int e = min(max(10 - ((int)(largest >> 23) - 127), -100), 123);
        const float up = __uint_as_float((uint32_t)(127 + e) << 23), down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int gi = 0; gi < G; ++gi) {
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                float x[8];
                unpack8<T>(raw[gi][w], x);
                // dimensions i and i + 4 together, as codes come out of a word; the even ones beside c 2^-24
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float f = i & 1 ? up : 16.0f * up;
                    const uint32_t held = Pair<__half>::pack(x[i] * f, x[i + 4] * f);
                    qf[gi][w][i >> 1][nt][i & 1] = held;
                    const float2 back = Pair<__half>::unpack(held);
                    sum += (back.x + back.y) * (i & 1 ? 0x1p-20f : 0x1p-24f);
                }
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            qsum[gi][nt][0] = __shfl_sync(0xffffffffu, sum, 8 * t);
            qsum[gi][nt][1] = __shfl_sync(0xffffffffu, sum, 8 * t + 4);
        }
        factor[nt][0] = plain * 0x1p20f * __shfl_sync(0xffffffffu, down, 8 * t);
        factor[nt][1] = plain * 0x1p20f * __shfl_sync(0xffffffffu, down, 8 * t + 4);
    }
    __syncthreads();

    // ---- the warp's chunks
    float o[G][4][NT][4], base[NT][2], l[NT][2], mid[G][NT][2];     // sums of 2^(score - base)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            base[nt][e] = -3.402823466e38f;
            l[nt][e] = 0.0f;
#pragma unroll
            for (int gi = 0; gi < G; ++gi) mid[gi][nt][e] = 0.0f;
        }
#pragma unroll
        for (int gi = 0; gi < G; ++gi)
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[gi][i][nt][e] = 0.0f;
    }
    const uint32_t factors = t4_smem(smem) + C::RING + warp * C::FACTORS;
    const int whole = min(ctx, n);                         // keys below it are seen by all, where their pages are there
    int stage = 0;
#pragma unroll 1
    for (int chunk = first; chunk < chunks; chunk += step) {
        copies_wait<C::STAGES - 2>();
        __syncwarp();
        // the next copy takes the stage that was read in the last turn
        const uint32_t there = __ballot_sync(0xffffffffu, there_is(pages[0]));          // bit 8 i: the page of keys 8 i on
        const int ahead = chunk + (C::STAGES - 1) * step;
        if (ahead < chunks) copy(ahead, stage == 0 ? C::STAGES - 1 : stage - 1, pages[C::STAGES - 1]);
        copies_commit();
#pragma unroll
        for (int i = 0; i < C::STAGES; ++i) pages[i] = pages[i + 1];
        pages[C::STAGES] = look_up(chunk + (C::STAGES + 1) * step);
        const uint32_t at = ring + stage * C::STAGE;
        const bool full = (chunk + 1) * kT4Keys <= whole && there == 0xffffffffu;
        key_factors<T, D>(at + 2 * kT4Keys * C::CODES, at + 2 * kT4Keys * C::CODES + kT4Keys * C::PARAMS, factors, lane);

        // scores in log2 units: of keys 16 mt + 2 g (c0, c1) and the next one (c2, c3)
        float z[2][NT][4];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
            float acc[G][NT][4];
            const int k0 = 16 * mt + 2 * g, k1 = k0 + 1;
#pragma unroll
            for (int gi = 0; gi < G; ++gi) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[gi][nt][e] = 0.0f;
                const uint2 x = lds64(at + code_at<D>(k0, 2 * gi + (t >> 1)) + 8 * (t & 1));
                const uint2 y = lds64(at + code_at<D>(k1, 2 * gi + (t >> 1)) + 8 * (t & 1));
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const uint32_t xw = w ? x.y : x.x, yw = w ? y.y : y.x;
                    const uint32_t x8 = xw >> 8, y8 = yw >> 8;
                    const uint32_t a0 = codes_low(xw), a1 = codes_low(yw), a2 = codes_high(xw), a3 = codes_high(yw);
                    const uint32_t b0 = codes_low(x8), b1 = codes_low(y8), b2 = codes_high(x8), b3 = codes_high(y8);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma_16x8x16(acc[gi][nt], a0, a1, a2, a3, qf[gi][w][0][nt][0], qf[gi][w][0][nt][1]);
                        mma_16x8x16(acc[gi][nt], b0, b1, b2, b3, qf[gi][w][1][nt][0], qf[gi][w][1][nt][1]);
                    }
                }
            }
            float s0[G], m0[G], s1[G], m1[G];
            factors_k<D>(factors, 16 * mt + g, s0, m0);
            factors_k<D>(factors, 16 * mt + 8 + g, s1, m1);
#pragma unroll
            for (int gi = 0; gi < G; ++gi)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {       // two queries at once
                        const float s = e < 2 ? s0[gi] : s1[gi], m = e < 2 ? m0[gi] : m1[gi];
                        float(&x)[4] = z[mt][nt];
                        if (gi) ffma2(x[e], x[e + 1], m, m, qsum[gi][nt][0], qsum[gi][nt][1], x[e], x[e + 1]);
                        else fmul2(x[e], x[e + 1], m, m, qsum[gi][nt][0], qsum[gi][nt][1]);
                        ffma2(x[e], x[e + 1], s, s, acc[gi][nt][e], acc[gi][nt][e + 1], x[e], x[e + 1]);
                    }
        }
        float ratio[4][G], centre[4][G], log_s[4], inv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) factors_v<D>(factors, 8 * i + g, ratio[i], centre[i], log_s[i], inv[i]);
        if (p.score.cap_out != 0.0f) {                     // cap tanh(x / cap), tanh(x) = 1 - 2 / (1 + e^2x)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float& x = z[i >> 1][nt][2 * (i & 1) + e];
                        x = fmaf(p.score.cap_out, 1.0f - __fdividef(2.0f, 1.0f + exp2_fast(x * factor[nt][e])), log_s[i]);
                    }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float* x = &z[i >> 1][nt][2 * (i & 1)];
                    ffma2(x[0], x[1], x[0], x[1], factor[nt][0], factor[nt][1], log_s[i], log_s[i]);
                }
        }
        uint32_t hidden = 0u;                              // bit 4 (2 mt + e / 2) + 2 nt + e % 2: the query does not see the key
        if (!full) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = 16 * (i >> 1) + 2 * g + (i & 1), j = chunk * kT4Keys + k;
                const bool real = j < n && (there >> (k & 24) & 1u);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int node = min((tile * C::ROWS + 8 * nt + 2 * t + e) / p.group, nodes - 1);
                        const bool sees = real && (j < ctx || (j - ctx < nodes && (sh.sees[node] >> (j - ctx) & 1ull)));
                        if (!sees) {
                            hidden |= 1u << (4 * i + 2 * nt + e);
                            z[i >> 1][nt][2 * (i & 1) + e] = -INFINITY;
                        }
                    }
            }
        }

        // The base moves only where a score is 2^8 above what it was set for: 2^6 below the largest then, so that p s
        // stays under 2^14 and what is 2^-20 of the largest is still a normal fp16.
        float top[NT][2];
        bool grew = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                top[nt][e] = fmaxf(fmaxf(z[0][nt][e], z[0][nt][2 + e]), fmaxf(z[1][nt][e], z[1][nt][2 + e]));
                grew |= top[nt][e] > base[nt][e] + 14.0f;
            }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int s = 4; s < 32; s <<= 1) top[nt][e] = fmaxf(top[nt][e], __shfl_xor_sync(0xffffffffu, top[nt][e], s));
                    // by the query's own scores alone: no other query has a say in its roundings
                    const float next = top[nt][e] > base[nt][e] + 14.0f ? top[nt][e] - 6.0f : base[nt][e], f = exp2_fast(base[nt][e] - next);
                    base[nt][e] = next;
                    l[nt][e] *= f;
#pragma unroll
                    for (int gi = 0; gi < G; ++gi) {
                        mid[gi][nt][e] *= f;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            o[gi][i][nt][e] *= f;
                            o[gi][i][nt][2 + e] *= f;
                        }
                    }
                }
        }

        uint32_t pf[G][2][NT][2];                          // p s, the second product's second operand
        auto weigh = [&](auto masked) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float* x = &z[i >> 1][nt][2 * (i & 1)];
                    fadd2(x[0], x[1], -base[nt][0], -base[nt][1]);
                    x[0] = exp2_fast(x[0]);
                    x[1] = exp2_fast(x[1]);
                    ffma2(l[nt][0], l[nt][1], x[0], x[1], inv[i], inv[i], l[nt][0], l[nt][1]);
#pragma unroll
                    for (int gi = 0; gi < G; ++gi) {
                        float w[2], c[2] = {centre[i][gi], centre[i][gi]};
                        fmul2(w[0], w[1], x[0], x[1], ratio[i][gi], ratio[i][gi]);
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (decltype(masked)::value && (hidden >> (4 * i + 2 * nt + e) & 1u)) w[e] = c[e] = 0.0f;      // whatever its scale holds
                        ffma2(mid[gi][nt][0], mid[gi][nt][1], x[0], x[1], c[0], c[1], mid[gi][nt][0], mid[gi][nt][1]);
                        pf[gi][i >> 1][nt][i & 1] = transpose8(Pair<__half>::pack(w[0], w[1]));
                    }
                }
            }
        };
        if (full) weigh(std::false_type{});
        else weigh(std::true_type{});

        // O^T += codes^T p: product i of a group has dimensions 16 i + 2 g (c0, c1) and the next one (c2, c3) as rows
        // the 8 leaves with the sum of what was rounded, a product with ones
        constexpr uint32_t ONE = 0x3c003c00u;
        const uint32_t vc = at + kT4Keys * C::CODES;
#pragma unroll
        for (int gi = 0; gi < G; ++gi) {
            float sums[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int e = 0; e < 4; ++e) sums[nt][e] = 0.0f;
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) mma_16x8x16(sums[nt], ONE, ONE, ONE, ONE, pf[gi][mt][nt][0], pf[gi][mt][nt][1]);
            }
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                uint32_t v[4];
                load_transposed(v, vc + code_at<D>(16 * mt + (lane & 15), 2 * gi + (lane >> 4)));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint32_t p0 = pf[gi][mt][nt][0], p1 = pf[gi][mt][nt][1];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mma_16x8x16(o[gi][i][nt], codes_low(v[i]), codes_high(v[i]), codes_low(v[i] >> 8), codes_high(v[i] >> 8), p0, p1);
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float(&x)[4] = o[gi][i][nt];
                    ffma2(x[0], x[1], sums[nt][0], sums[nt][1], -0x1p-21f, -0x1p-21f, x[0], x[1]);
                    ffma2(x[2], x[3], sums[nt][2], sums[nt][3], -0x1p-17f, -0x1p-17f, x[2], x[3]);
                }
        }

        stage = stage == C::STAGES - 1 ? 0 : stage + 1;
    }
    copies_wait<0>();

    // ---- the warps' states, joined in the ring
    float* state = reinterpret_cast<float*>(smem);
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int s = 4; s < 32; s <<= 1) {
                l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], s);
#pragma unroll
                for (int gi = 0; gi < G; ++gi) mid[gi][nt][e] += __shfl_xor_sync(0xffffffffu, mid[gi][nt][e], s);
            }
            float* to = state + warp * C::PART + (8 * nt + 2 * t + e) * C::PITCH;
            if (g == 0) {
                to[0] = l[nt][e] == 0.0f ? -INFINITY : base[nt][e];
                to[1] = l[nt][e];
            }
#pragma unroll
            for (int gi = 0; gi < G; ++gi) {
                const float back = mid[gi][nt][e];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<float2*>(to + 2 + 64 * gi + 16 * i + 2 * g) =
                        make_float2(fmaf(o[gi][i][nt][e], 0x1p24f, back), fmaf(o[gi][i][nt][2 + e], 0x1p20f, back));
            }
        }
    __syncthreads();
    constexpr int PAIRS = D / 2;
    auto write = [&](int q, int d, float x, float y, float sum) {
        const int r = tile * C::ROWS + q, node = r / p.group;
        if (r >= rows) return;
        const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
        T* out = static_cast<T*>(p.O) + (q0 + node) * p.o_row + (h * p.group + r % p.group) * p.o_head + d;
        *reinterpret_cast<uint32_t*>(out) = Pair<T>::pack(x * f, y * f);
    };
    for (int i = threadIdx.x; i < C::ROWS * PAIRS; i += kT4Threads) {
        const int q = i / PAIRS, d = 2 * (i % PAIRS);
        float most, sum;
        float2 v;
        t4_join<C>([&](int i, int at) { return state[i * C::PART + at]; }, kT4Warps, q, d, most, sum, v);
        out(write, q, d, most, sum, v);
    }
    return true;
}

template <class C>
__global__ void __launch_bounds__(kT4Threads, C::CTAS)
    gsr_tree4_cluster_kernel(const __grid_constant__ Tree4Params p, const __grid_constant__ Tree4Plan plan) {
    extern __shared__ __align__(128) char smem[];
    __shared__ T4Shared sh;
    constexpr int PAIRS = C::D / 2;
    const int rank = blockIdx.x % plan.cluster, item = blockIdx.x / plan.cluster;
    const int tile = item % plan.tiles, h = item / plan.tiles % p.Hkv, b = item / plan.tiles / p.Hkv;
    float* mine = reinterpret_cast<float*>(smem) + kT4Warps * C::PART;
    const bool some = t4_part<C>(p, plan, smem, sh, b, h, tile, rank + plan.cluster * (threadIdx.x >> 5), plan.cluster * kT4Warps, INT_MAX,
               [&](auto write, int q, int d, float most, float sum, float2 v) {
                   if (plan.cluster == 1) {
                       write(q, d, v.x, v.y, sum);
                       return;
                   }
                   if (d == 0) *reinterpret_cast<float2*>(mine + q * C::PITCH) = make_float2(most, sum);
                   *reinterpret_cast<float2*>(mine + q * C::PITCH + 2 + d) = v;
               });
    if (plan.cluster == 1 || !some) return;                 // the whole cluster
    // ---- over the cluster, each CTA a share of the outputs
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    const T4Request req = t4_request<C::ROWS>(p, b);
    const uint32_t here = t4_smem(mine);
    for (int i = rank * kT4Threads + threadIdx.x; i < C::ROWS * PAIRS; i += plan.cluster * kT4Threads) {
        const int q = i / PAIRS, d = 2 * (i % PAIRS), r = tile * C::ROWS + q;
        // all of the states at once: one trip to the other CTAs
        float2 ms[kT4MaxCluster], v[kT4MaxCluster];
#pragma unroll
        for (int k = 0; k < kT4MaxCluster; ++k) {
            ms[k] = make_float2(-INFINITY, 0.0f);
            v[k] = make_float2(0.0f, 0.0f);
            if (k < plan.cluster) {
                uint32_t a;
                asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(here + 4 * q * C::PITCH), "r"(k));
                asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(ms[k].x), "=f"(ms[k].y) : "r"(a) : "memory");
                asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v[k].x), "=f"(v[k].y) : "r"(a + 8 + 4 * d) : "memory");
            }
        }
        float most = -INFINITY, sum = 0.0f;
        float2 o = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < kT4MaxCluster; ++k) most = fmaxf(most, ms[k].x);
#pragma unroll
        for (int k = 0; k < kT4MaxCluster; ++k) {
            if (ms[k].x == -INFINITY) continue;
            const float f = exp2_fast(ms[k].x - most);
            sum = fmaf(f, ms[k].y, sum);
            o.x = fmaf(f, v[k].x, o.x);
            o.y = fmaf(f, v[k].y, o.y);
        }
        if (r >= req.rows) continue;
        const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
        typename C::T* to = static_cast<typename C::T*>(p.O) + (req.q0 + r / p.group) * p.o_row + (h * p.group + r % p.group) * p.o_head + d;
        *reinterpret_cast<uint32_t*>(to) = Pair<typename C::T>::pack(o.x * f, o.y * f);
    }
    // no CTA leaves while another reads its states
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Of a grid's CTAs as many take part as have eight units, two chunks a warp, or one.  CTA c's first unit of U, and the CTA that holds unit u.
__device__ __forceinline__ int t4_busy(long long U, int grid) { return (int)max(min(U / 8, (long long)grid), min(U, 1ll)); }
__device__ __forceinline__ long long t4_first(long long U, int c, int G) { return U * c / G; }
__device__ __forceinline__ int t4_cta_of(long long U, long long u, int G) { return (int)(((u + 1) * G - 1) / U); }

template <class C>
__global__ void __launch_bounds__(kT4Threads, C::CTAS)
    gsr_tree4_even_kernel(const __grid_constant__ Tree4Params p, const __grid_constant__ Tree4Plan plan) {
    extern __shared__ __align__(128) char smem[];
    __shared__ T4Shared sh;
    __shared__ long long s_sums[kT4Warps], s_first[2];
    grid_launch_next();                                     // the joining CTAs, as SMs fall free
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // ---- this CTA's range of units
    const int per = (p.B + kT4Threads - 1) / kT4Threads, b0 = min((int)threadIdx.x * per, p.B), b1 = min(b0 + per, p.B);
    long long sum = 0;
    for (int b = b0; b < b1; ++b) sum += t4_request<C::ROWS>(p, b).units(p.Hkv);
    long long upto = sum;                                   // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) s_sums[warp] = upto;
    __syncthreads();
    long long U = 0;
#pragma unroll
    for (int i = 0; i < kT4Warps; ++i) {
        if (i < warp) upto += s_sums[i];
        U += s_sums[i];
    }
    const int busy = t4_busy(U, gridDim.x);
    const bool takes = (int)blockIdx.x < busy;
    const long long u_begin = takes ? t4_first(U, blockIdx.x, busy) : U, u_end = takes ? t4_first(U, blockIdx.x + 1, busy) : U;
    long long before = upto - sum;
    for (int b = b0; b < b1; ++b) {
        const long long units = t4_request<C::ROWS>(p, b).units(p.Hkv);
        if (blockIdx.x == 0) p.unit_starts[b] = before;     // for the joining launch
        if (before <= u_begin && u_begin < before + units) {
            s_first[0] = b;
            s_first[1] = u_begin - before;
        }
        before += units;
    }
    if (blockIdx.x == 0 && threadIdx.x == kT4Threads - 1) p.unit_starts[p.B] = U;
    __syncthreads();
    int b = takes ? (int)s_first[0] : p.B;
    long long off = takes ? s_first[1] : 0;
    for (long long u = u_begin; u < u_end && b < p.B;) {
        const T4Request req = t4_request<C::ROWS>(p, b);
        if (off >= req.units(p.Hkv)) {                      // the range goes on in a later request
            off = 0;
            ++b;
            continue;
        }
        const int chunks = max(req.chunks, 1), index = (int)(off / chunks), h = index / req.tiles, tile = index - h * req.tiles;
        const int c0 = (int)(off - (long long)index * chunks), c1 = (int)min((long long)chunks, c0 + (u_end - u));
        const bool all = c0 == 0 && c1 == chunks;
        float* slot = p.parts + (2ll * blockIdx.x + (u > u_begin ? 1 : 0)) * C::PART;
        t4_part<C>(p, plan, smem, sh, b, h, tile, c0 + warp, kT4Warps, c1, [&](auto write, int q, int d, float most, float sum, float2 v) {
            if (all) {
                write(q, d, v.x, v.y, sum);
                return;
            }
            if (d == 0) *reinterpret_cast<float2*>(slot + q * C::PITCH) = make_float2(most, sum);
            *reinterpret_cast<float2*>(slot + q * C::PITCH + 2 + d) = v;
        });
        u += c1 - c0;
        off += c1 - c0;
        __syncthreads();                                    // the states have been read: the ring is free
    }
}

// A query row and head of an item that several CTAs share, by WARPS warps: the states in the order of the CTAs, warp by
// warp, then the warps'.
template <class C, int WARPS>
__global__ void __launch_bounds__(128) gsr_tree4_join_kernel(const __grid_constant__ Tree4Params p, int grid) {
    using T = typename C::T;
    constexpr int D = C::D, E = D / 32, ROWS = 4 / WARPS, AHEAD = WARPS > 1 ? 8 : 4;
    __shared__ float sm[4][D + 2];
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % WARPS;
    const long long id = (long long)blockIdx.x * ROWS + (threadIdx.x >> 5) / WARPS;
    const int row = (int)min(id / p.Hq, (long long)p.total_q), h = (int)(id % p.Hq), hk = h / p.group;
    int left = 0, right = p.B;                              // first request that ends behind the row
    while (left < right) {
        const int mid = (left + right) >> 1;
        if (__ldg(p.q_starts + mid + 1) <= row) left = mid + 1;
        else right = mid;
    }
    const int b = min(left, p.B - 1);
    const T4Request req = t4_request<C::ROWS>(p, b);
    const int t = row - req.q0, r = t * p.group + h - hk * p.group, tile = r / C::ROWS, chunks = max(req.chunks, 1);
    grid_wait();                                            // every CTA: this launch then ends after the parts'
    bool mine = row < p.total_q && left < p.B && t >= 0 && t < req.nodes;
    int c0 = 0, c1 = 0;
    bool starts_later = false;                              // the item does, than its first CTA's range
    const long long U = p.unit_starts[p.B];
    const int busy = t4_busy(U, grid);
    if (mine) {
        const long long s = p.unit_starts[b] + ((long long)hk * req.tiles + tile) * chunks;
        c0 = max(t4_cta_of(U, s, busy), 0);
        c1 = min(t4_cta_of(U, s + chunks - 1, busy), busy - 1);
        mine = c0 < c1;                                     // else written whole
        starts_later = t4_first(U, c0, busy) < s;
    }
    float m = -INFINITY, l = 0.0f, acc[E] = {};
    auto add = [&](float pm, float pl, const float* o) {
        if (pm == -INFINITY) return;                        // saw nothing
        const float next = fmaxf(m, pm), f0 = m == -INFINITY ? 0.0f : exp2_fast(m - next), f1 = exp2_fast(pm - next);
        l = m == -INFINITY ? pl * f1 : l * f0 + pl * f1;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = m == -INFINITY ? o[e] * f1 : acc[e] * f0 + o[e] * f1;
        m = next;
    };
    if (mine)
        for (int first = c0 + warp; first <= c1; first += WARPS * AHEAD) {
            float2 ml[AHEAD];
            float x[AHEAD][E];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {               // all loads, then the sums in order
                const int c = first + k * WARPS;
                ml[k] = make_float2(-INFINITY, 0.0f);
                if (c > c1) continue;
                // an item that starts behind the CTA's first unit has its second slot
                const float* at = p.parts + (2ll * c + (c == c0 && starts_later ? 1 : 0)) * C::PART + (r - tile * C::ROWS) * C::PITCH;
                ml[k] = *reinterpret_cast<const float2*>(at);
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    const float2 v = *reinterpret_cast<const float2*>(at + 2 + lane * E + e);
                    x[k][e] = v.x;
                    x[k][e + 1] = v.y;
                }
            }
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) add(ml[k].x, ml[k].y, x[k]);
        }
    if (WARPS > 1) {
#pragma unroll
        for (int e = 0; e < E; ++e) sm[warp][lane * E + e] = acc[e];
        if (lane == 0) {
            sm[warp][D] = m;
            sm[warp][D + 1] = l;
        }
        __syncthreads();
        if (warp != 0) return;
#pragma unroll
        for (int i = 1; i < WARPS; ++i) add(sm[i][D], sm[i][D + 1], &sm[i][lane * E]);
    }
    if (!mine) return;
    const float f = l == 0.0f ? 0.0f : 1.0f / l;
    uint32_t* to = reinterpret_cast<uint32_t*>(static_cast<T*>(p.O) + row * p.o_row + h * p.o_head + lane * E);
#pragma unroll
    for (int e = 0; e < E; e += 2) to[e / 2] = Pair<T>::pack(acc[e] * f, acc[e + 1] * f);
}

// Shared memory that a kernel may use, said once a device.
template <class K>
cudaError_t t4_allow(K kernel, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev <= 63 && (done.load(std::memory_order_acquire) >> dev & 1))) return e;
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) != cudaSuccess) return e;
    if (dev <= 63) done.fetch_or(1ull << dev, std::memory_order_release);
    return cudaSuccess;
}

template <class C>
cudaError_t launch_tree4_cfg(const Tree4Params& p, const Tree4Split& split, cudaStream_t stream) {
    static std::atomic<uint64_t> cluster_done{0}, even_done{0};
    static_assert(C::ROWS == 8 * C::NT && C::PART * 4 == Tree4Split::state_bytes(C::NT, C::D), "");
    cudaError_t e;
    const Tree4Plan plan{Divider((uint32_t)p.page), split.tiles, split.cluster, split.chunks};
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr;
    cfg.gridDim = dim3((unsigned)split.grid);
    cfg.blockDim = dim3(kT4Threads);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    if (split.cluster) {
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = (unsigned)split.cluster;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        if ((e = t4_allow(gsr_tree4_cluster_kernel<C>, C::SMEM, cluster_done)) != cudaSuccess) return e;
        return cudaLaunchKernelEx(&cfg, gsr_tree4_cluster_kernel<C>, p, plan);
    }
    if ((e = t4_allow(gsr_tree4_even_kernel<C>, C::SMEM, even_done)) != cudaSuccess ||
        (e = cudaLaunchKernelEx(&cfg, gsr_tree4_even_kernel<C>, p, plan)) != cudaSuccess)
        return e;
    // the joining CTAs start while the parts' last CTAs finish, and wait for them there
    // eight states an item or more by four warps a row, few by one
    const long long rows = (long long)p.total_q * p.Hq, items = (long long)p.B * p.Hkv * split.tiles;
    const bool many = split.grid >= 8 * items;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = 0;
    cfg.gridDim = dim3((unsigned)(many ? rows : (rows + 3) / 4));
    return many ? cudaLaunchKernelEx(&cfg, gsr_tree4_join_kernel<C, 4>, p, split.grid)
                : cudaLaunchKernelEx(&cfg, gsr_tree4_join_kernel<C, 1>, p, split.grid);
}

template <class T>
cudaError_t launch_tree4_type(const Tree4Params& p, const Tree4Split& split, cudaStream_t stream) {
    if (p.D == 64) return split.nt == 2 ? launch_tree4_cfg<T4Cfg<T, 64, 2>>(p, split, stream) : launch_tree4_cfg<T4Cfg<T, 64, 1>>(p, split, stream);
    return split.nt == 2 ? launch_tree4_cfg<T4Cfg<T, 128, 2>>(p, split, stream) : launch_tree4_cfg<T4Cfg<T, 128, 1>>(p, split, stream);
}

}  // namespace
}  // namespace gsr
