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
// does to O) leaves by a product with the constant, chunk by chunk: products are many fewer than values, and left
// to the end it would cost digits (4096 keys, fp16: 3.1e-4 of O).  Queries are held
// as fp16 times a power of two for each row (bf16's 8 bits fit; what is 2^-25 of the row's largest loses digits).
//
// What bounds it: D / 2 + D / 16 bytes a key and head, twice, from HBM; per byte that is 3.6 times the
// arithmetic of a 16-bit cache, so the instructions that unpack codes come next.  Codes are therefore unpacked
// in registers into mma.sync operands: operands of tcgen05 come from shared memory or TMEM, and the unpacked rows
// would be written there and read again, 93 of an SM's 128 bytes a clock at HBM's rate, before the first product.
// Keys are the products' rows (16 at once) and the queries of a group their columns (8): no row of the product is
// spent on padding where a group has 4 or 8 heads.
//
// Split: a cluster of CTAs shares the keys of one request, head and tile of 8 NT query rows, in chunks of 32
// that warps take in turn; each warp copies its own chunks (cp.async, three in flight), with its own softmax
// state.  States are joined in shared memory, over the cluster by distributed shared memory: one launch, no
// workspace, no order that changes.
#pragma once

#include <atomic>
#include <type_traits>

#include "gsr.h"
#include "rows16.cuh"
#include "serving.h"

namespace gsr {
namespace {

constexpr int kT4Warps = 4, kT4Threads = 32 * kT4Warps, kT4Keys = 32;

struct Tree4Plan {
    Divider by_page;
    int tiles;                  // tiles of query rows a request and head
    int cluster;
    int chunks;                 // that a table's row can hold
};

template <class Type, int Dim, int Nt>
struct T4Cfg {
    using T = Type;
    static constexpr int D = Dim, NT = Nt, G = D / 64, ROWS = 8 * NT;
    static constexpr int STAGES = NT == 1 ? 2 : 3;
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

template <class C>
__global__ void __launch_bounds__(kT4Threads, C::NT == 1 ? 4 : 2)
    gsr_tree4_kernel(const __grid_constant__ Tree4Params p, const __grid_constant__ Tree4Plan plan) {
    using T = typename C::T;
    constexpr int D = C::D, G = C::G, NT = C::NT;
    extern __shared__ __align__(128) char smem[];
    __shared__ uint64_t s_sees[GSR_TREE_MAX_NODES];
    __shared__ int s_parent[GSR_TREE_MAX_NODES];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int rank = blockIdx.x % plan.cluster, item = blockIdx.x / plan.cluster;
    const int tile = item % plan.tiles, h = item / plan.tiles % p.Hkv, b = item / plan.tiles / p.Hkv;

    const int* table = p.table + (long long)b * p.table_width;
    const int q0 = __ldg(p.q_starts + b), q1 = __ldg(p.q_starts + b + 1), kv = __ldg(p.kv_lens + b);

    // ---- the pages of a chunk: eight keys lie in one; a lane looks after keys 8 (lane / 8) on
    const int part = lane >> 3, j8 = lane & 7;
    const int step = plan.cluster * kT4Warps, first = rank + plan.cluster * warp;
    auto look_up = [&](int chunk) {                         // whatever the length is: entries of the table are there
        const int col = plan.by_page(min(chunk, plan.chunks) * kT4Keys + 8 * part);
        return col < p.table_width ? __ldg(table + col) : -1;
    };
    int pages[C::STAGES + 1];                               // of the chunks in flight, and of the next two
#pragma unroll
    for (int i = 0; i <= C::STAGES; ++i) pages[i] = look_up(first + i * step);

    const int drafted = q1 - q0, nodes = q0 < 0 ? 0 : min(min(drafted, p.max_nodes), p.total_q - q0), rows = nodes * p.group;
    if (tile * C::ROWS >= rows) return;                                     // the whole cluster
    const int ctx = kv - drafted;                                           // keys before the tree
    const int n = (int)min((long long)kv, (long long)p.table_width * p.page), chunks = n > 0 ? (n + kT4Keys - 1) / kT4Keys : 0;

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

    // ---- which nodes see which: bit u of s_sees[t]
    if (threadIdx.x < nodes) s_parent[threadIdx.x] = p.parents ? __ldg(p.parents + q0 + threadIdx.x) : (int)threadIdx.x - 1;
    __syncthreads();
    if (threadIdx.x < nodes) {
        int u = threadIdx.x;
        uint64_t bits = 1ull << u;
        if (!p.parents) bits = bits * 2 - 1;
        else
            for (int up = s_parent[u]; up >= 0 && up < u; up = s_parent[u]) {
                bits |= 1ull << up;
                u = up;
            }
        s_sees[threadIdx.x] = bits;
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
        // the row times 2^e is below 2^11 beside c 2^-20, and 16 times that beside c 2^-24
        const int e = min(max(10 - ((int)(largest >> 23) - 127), -100), 100);
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
                    for (int e = 0; e < 4; ++e) {
                        const float s = e < 2 ? s0[gi] : s1[gi], m = e < 2 ? m0[gi] : m1[gi];
                        const float x = gi ? fmaf(m, qsum[gi][nt][e & 1], z[mt][nt][e]) : m * qsum[gi][nt][e & 1];
                        z[mt][nt][e] = fmaf(s, acc[gi][nt][e], x);
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
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float& x = z[i >> 1][nt][2 * (i & 1) + e];
                        x = fmaf(x, factor[nt][e], log_s[i]);
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
                        const bool sees = real && (j < ctx || (j - ctx < nodes && (s_sees[node] >> (j - ctx) & 1ull)));
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
                    const float next = fmaxf(base[nt][e], top[nt][e] - 6.0f), f = exp2_fast(base[nt][e] - next);
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
                    float w[G][2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float x = exp2_fast(z[i >> 1][nt][2 * (i & 1) + e] - base[nt][e]);
                        l[nt][e] = fmaf(x, inv[i], l[nt][e]);
                        const bool out = decltype(masked)::value && (hidden >> (4 * i + 2 * nt + e) & 1u);     // whatever its scale holds
#pragma unroll
                        for (int gi = 0; gi < G; ++gi) {
                            w[gi][e] = out ? 0.0f : x * ratio[i][gi];
                            mid[gi][nt][e] = out ? mid[gi][nt][e] : fmaf(x, centre[i][gi], mid[gi][nt][e]);
                        }
                    }
#pragma unroll
                    for (int gi = 0; gi < G; ++gi) pf[gi][i >> 1][nt][i & 1] = transpose8(Pair<__half>::pack(w[gi][0], w[gi][1]));
                }
            }
        };
        if (full) weigh(std::false_type{});
        else weigh(std::true_type{});

        // O^T += codes^T p: product i of a group has dimensions 16 i + 2 g (c0, c1) and the next one (c2, c3) as rows
        constexpr uint32_t LOW8 = 0x80088008u, HIGH8 = 0x80808080u;         // -8 as the codes are held
        const uint32_t vc = at + kT4Keys * C::CODES;
#pragma unroll
        for (int gi = 0; gi < G; ++gi)
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                uint32_t v[4];
                load_transposed(v, vc + code_at<D>(16 * mt + (lane & 15), 2 * gi + (lane >> 4)));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint32_t p0 = pf[gi][mt][nt][0], p1 = pf[gi][mt][nt][1];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        mma_16x8x16(o[gi][i][nt], codes_low(v[i]), codes_high(v[i]), codes_low(v[i] >> 8), codes_high(v[i] >> 8), p0, p1);
                        mma_16x8x16(o[gi][i][nt], LOW8, HIGH8, LOW8, HIGH8, p0, p1);
                    }
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
    // states of row q from `count` places, each state_of(i)[...]: largest M, and sums weighed by 2^(M_i - M)
    auto join = [&](auto state_of, int count, int q, int d, float& most, float& sum, float2& v) {
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
    };
    auto of_warp = [&](int i, int at) { return state[i * C::PART + at]; };
    float* mine = state + kT4Warps * C::PART;
    for (int i = threadIdx.x; i < C::ROWS * PAIRS; i += kT4Threads) {
        const int q = i / PAIRS, d = 2 * (i % PAIRS);
        float most, sum;
        float2 v;
        join(of_warp, kT4Warps, q, d, most, sum, v);
        if (plan.cluster == 1) write(q, d, v.x, v.y, sum);
        else {
            if (d == 0) {
                mine[q * C::PITCH] = most;
                mine[q * C::PITCH + 1] = sum;
            }
            *reinterpret_cast<float2*>(mine + q * C::PITCH + 2 + d) = v;
        }
    }
    if (plan.cluster == 1) return;
    // ---- and over the cluster, each CTA a share of the outputs
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    const uint32_t here = t4_smem(mine);
    auto of_cta = [&](int i, int at) {
        uint32_t a;
        float x;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(here + 4 * at), "r"(i));
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(a) : "memory");
        return x;
    };
    for (int i = rank * kT4Threads + threadIdx.x; i < C::ROWS * PAIRS; i += plan.cluster * kT4Threads) {
        const int q = i / PAIRS, d = 2 * (i % PAIRS);
        float most, sum;
        float2 v;
        join(of_cta, plan.cluster, q, d, most, sum, v);
        write(q, d, v.x, v.y, sum);
    }
    // no CTA leaves while another reads its states
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <class C>
cudaError_t launch_tree4_cfg(const Tree4Params& p, int sms, cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};                  // devices whose kernel has its shared memory
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev > 63 || !(done.load(std::memory_order_acquire) >> dev & 1)) {
        if ((e = cudaFuncSetAttribute(gsr_tree4_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM)) != cudaSuccess) return e;
        if (dev <= 63) done.fetch_or(1ull << dev, std::memory_order_release);
    }
    Tree4Plan plan{Divider((uint32_t)p.page), (p.max_nodes * p.group + C::ROWS - 1) / C::ROWS, 1, 0};
    const long long items = (long long)p.B * p.Hkv * plan.tiles;
    const long long chunks = ((long long)p.table_width * p.page + kT4Keys - 1) / kT4Keys;
    plan.chunks = (int)chunks;
    while (plan.cluster < 8 && items * plan.cluster < 8ll * sms && chunks > (long long)plan.cluster * kT4Warps) plan.cluster *= 2;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)plan.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(items * plan.cluster));
    cfg.blockDim = dim3(kT4Threads);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gsr_tree4_kernel<C>, p, plan);
}

template <class T>
cudaError_t launch_tree4_type(const Tree4Params& p, int sms, cudaStream_t stream) {
    const bool wide = p.max_nodes * p.group > 8;           // more rows than one column tile holds
    if (p.D == 64) return wide ? launch_tree4_cfg<T4Cfg<T, 64, 2>>(p, sms, stream) : launch_tree4_cfg<T4Cfg<T, 64, 1>>(p, sms, stream);
    return wide ? launch_tree4_cfg<T4Cfg<T, 128, 2>>(p, sms, stream) : launch_tree4_cfg<T4Cfg<T, 128, 1>>(p, sms, stream);
}

}  // namespace
}  // namespace gsr
