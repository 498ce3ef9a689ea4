// attention_tree4.cuh - attention of drafted tokens over a paged cache of 4 bits (one token a request is
// ordinary decoding).
//
// A key (value) is s code + m for each 64 of its dimensions, so with the codes c and C of a key and a value
//   score_j = sum_g s_jg (q_g . (c_jg - 8)) + (m_jg + 8 s_jg) sum(q_g),
//   O = sum_j p_j s_jg (C_jg - 8) + sum_j p_j (m_jg + 8 s_jg):
// both products run on the codes themselves, which 16-bit types hold exactly, and scales and minima are applied to
// their results and to p, in fp32.
//
// What bounds it: D / 2 + D / 16 bytes a key and head, twice, from HBM; per byte that is 5.7 times the
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

#include "gsr.h"
#include "rows16.cuh"
#include "serving.h"

namespace gsr {
namespace {

constexpr int kT4Warps = 8, kT4Threads = 32 * kT4Warps, kT4Stages = 3, kT4Keys = 32;

struct Tree4Plan {
    Divider by_page;
    int tiles;                  // tiles of query rows a request and head
    int cluster;
};

template <class Type, int Dim, int Nt>
struct T4Cfg {
    using T = Type;
    static constexpr int D = Dim, NT = Nt, G = D / 64, ROWS = 8 * NT;
    static constexpr int CODES = D / 2, PARAMS = D / 16;             // bytes of a row
    static constexpr int STAGE = kT4Keys * 2 * (CODES + PARAMS);
    static constexpr int RING = kT4Warps * kT4Stages * STAGE;
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
template <class T>
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (Pair<T>::bf16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Codes i and i + 4 of a word less 8, as two operands: the code's bits in the mantissa of 64 (fp16) or 128 (bf16),
// and one exact subtraction.  (Left in the products, the offset costs digits where they cancel: the sums run to 72
// times a result that is a fraction of one.)
template <class T, int I>
__device__ __forceinline__ uint32_t codes_of(uint32_t w) {
    if constexpr (Pair<T>::bf16) {
        const uint32_t v = (w >> (4 * I) & 0x000f000fu) | 0x43004300u, c = 0x43084308u;
        const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), *reinterpret_cast<const __nv_bfloat162*>(&c));
        return *reinterpret_cast<const uint32_t*>(&r);
    } else {
        const uint32_t v = ((I ? w >> (I ? 4 * I - 4 : 0) : w << 4) & 0x00f000f0u) | 0x54005400u, c = 0x54805480u;
        const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&c));
        return *reinterpret_cast<const uint32_t*>(&r);
    }
}
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Where 16-byte piece c of key k's codes lies in a stage: rows that a warp reads at once (keys 0 to 3, or 0, 4, 1, 5
// of 8) meet in no bank.
template <int D>
__device__ __forceinline__ int code_at(int k, int c) {
    if constexpr (D == 128) return k * 64 + (c ^ ((k >> 1 ^ k >> 2) & 1) << 1) * 16;
    return (k ^ (k & 4) >> 1) * 32 + c * 16;
}

template <class C>
__global__ void __launch_bounds__(kT4Threads, C::NT == 1 ? 2 : 1)
    gsr_tree4_kernel(const __grid_constant__ Tree4Params p, const __grid_constant__ Tree4Plan plan) {
    using T = typename C::T;
    constexpr int D = C::D, G = C::G, NT = C::NT;
    extern __shared__ __align__(128) char smem[];
    __shared__ uint64_t s_sees[GSR_TREE_MAX_NODES];
    __shared__ int s_parent[GSR_TREE_MAX_NODES];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int rank = blockIdx.x % plan.cluster, item = blockIdx.x / plan.cluster;
    const int tile = item % plan.tiles, h = item / plan.tiles % p.Hkv, b = item / plan.tiles / p.Hkv;

    const int q0 = __ldg(p.q_starts + b), drafted = __ldg(p.q_starts + b + 1) - q0;
    const int nodes = q0 < 0 ? 0 : min(min(drafted, p.max_nodes), p.total_q - q0), rows = nodes * p.group;
    if (tile * C::ROWS >= rows) return;                                     // the whole cluster
    const int kv = __ldg(p.kv_lens + b), ctx = kv - drafted;               // keys before the tree
    const int n = (int)min((long long)kv, (long long)p.table_width * p.page), chunks = n > 0 ? (n + kT4Keys - 1) / kT4Keys : 0;
    const int* table = p.table + (long long)b * p.table_width;

    // ---- the copies of a chunk.  Eight keys lie in one page; lane i looks up that of keys 8 (i % 4) on.
    const uint32_t ring = t4_smem(smem) + warp * kT4Stages * C::STAGE;
    auto look_up = [&](int chunk, int& pg, int& row) {
        const int j = chunk * kT4Keys + 8 * (lane & 3);
        pg = -1;
        row = 0;
        if (chunk < chunks && j < n) {
            const int col = plan.by_page(j);
            row = j - col * p.page;
            pg = __ldg(table + col);
            if (pg < 0 || pg >= p.num_pages) pg = -1;
        }
    };
    auto copy = [&](int chunk, int stage, int pg, int row) {
        const uint32_t at = ring + stage * C::STAGE;
        constexpr int PIECES = C::CODES / 16, KEYS = 32 / PIECES;           // 16-byte pieces of a row, keys at once
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int k = i * KEYS + lane / PIECES, c = lane % PIECES;
            const int page = __shfl_sync(0xffffffffu, pg, k >> 3), r = __shfl_sync(0xffffffffu, row, k >> 3) + (k & 7);
            const bool real = page >= 0 && chunk * kT4Keys + k < n;
            const char* from_k = p.K.codes.data + page * p.K.codes.page + h * p.K.codes.head + r * p.K.codes.row + 16 * c;
            const char* from_v = p.V.codes.data + page * p.V.codes.page + h * p.V.codes.head + r * p.V.codes.row + 16 * c;
            copy_async<16>(at + code_at<D>(k, c), real ? from_k : p.Q, real);
            copy_async<16>(at + kT4Keys * C::CODES + code_at<D>(k, c), real ? from_v : p.Q, real);
        }
        const int page = __shfl_sync(0xffffffffu, pg, lane >> 3), r = __shfl_sync(0xffffffffu, row, lane >> 3) + (lane & 7);
        const bool real = page >= 0 && chunk * kT4Keys + lane < n;
        const char* from_k = p.K.params.data + page * p.K.params.page + h * p.K.params.head + r * p.K.params.row;
        const char* from_v = p.V.params.data + page * p.V.params.page + h * p.V.params.head + r * p.V.params.row;
        const uint32_t params = at + 2 * kT4Keys * C::CODES + lane * C::PARAMS;
        copy_async<C::PARAMS>(params, real ? from_k : p.Q, real);
        copy_async<C::PARAMS>(params + kT4Keys * C::PARAMS, real ? from_v : p.Q, real);
    };
    const int step = plan.cluster * kT4Warps, first = rank + plan.cluster * warp;
    int pages[kT4Stages], page_rows[kT4Stages];           // of the chunks in flight, and of the next one
#pragma unroll
    for (int i = 0; i < kT4Stages; ++i) look_up(first + i * step, pages[i], page_rows[i]);
#pragma unroll
    for (int i = 0; i < kT4Stages - 1; ++i) {
        if (first + i * step < chunks) copy(first + i * step, i, pages[i], page_rows[i]);
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

    // ---- queries: the products' second operand, columns n of 8, and their sums of each 64 dimensions
    uint32_t qf[G][2][2][NT][2];
    float qsum[G][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = tile * C::ROWS + 8 * nt + g, node = r / p.group;
        const T* q = static_cast<const T*>(p.Q) + (q0 + node) * p.q_row + (h * p.group + r % p.group) * p.q_head;
#pragma unroll
        for (int gi = 0; gi < G; ++gi) {
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (r < rows) v = *reinterpret_cast<const uint4*>(q + 64 * gi + 16 * t + 8 * w);
                const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = Pair<T>::unpack(x[i]);
                    sum += f.x + f.y;
                    // dimensions i and i + 4 together, as codes come out of a word
                    qf[gi][w][i >> 1][nt][i & 1] = __byte_perm(x[i >> 1], x[2 + (i >> 1)], i & 1 ? 0x7632 : 0x5410);
                }
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            qsum[gi][nt][0] = __shfl_sync(0xffffffffu, sum, 8 * t);
            qsum[gi][nt][1] = __shfl_sync(0xffffffffu, sum, 8 * t + 4);
        }
    }
    __syncthreads();

    // ---- the warp's chunks
    float o[G][4][NT][4], m[NT][2], l[NT][2], mid[G][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            m[nt][e] = -INFINITY;
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
    const int kappa = (g >> 1) + 4 * (g & 1);              // the key of 8 that row g of a product is
    const int whole = min(ctx, n);                         // keys below it are seen by all, where their pages are there
    int stage = 0;
#pragma unroll 1
    for (int chunk = first; chunk < chunks; chunk += step) {
        copies_wait<kT4Stages - 2>();
        __syncwarp();
        const uint32_t at = ring + stage * C::STAGE;
        const bool full = (chunk + 1) * kT4Keys <= whole && !__any_sync(0xffffffffu, pages[0] < 0);
        const uint32_t there = __ballot_sync(0xffffffffu, pages[0] >= 0);          // bit i: the page of keys 8 i on

        // scores in log2 units: rows of products 2 mt (c0, c1) and 2 mt + 1 (c2, c3) of 8 keys
        float z[2][NT][4];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
            float acc[G][NT][4];
            const int k0 = 16 * mt + kappa, k1 = k0 + 8;
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
                    const uint32_t a0 = codes_of<T, 0>(xw), a1 = codes_of<T, 0>(yw), a2 = codes_of<T, 1>(xw), a3 = codes_of<T, 1>(yw);
                    const uint32_t b0 = codes_of<T, 2>(xw), b1 = codes_of<T, 2>(yw), b2 = codes_of<T, 3>(xw), b3 = codes_of<T, 3>(yw);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma_16x8x16<T>(acc[gi][nt], a0, a1, a2, a3, qf[gi][w][0][nt][0], qf[gi][w][0][nt][1]);
                        mma_16x8x16<T>(acc[gi][nt], b0, b1, b2, b3, qf[gi][w][1][nt][0], qf[gi][w][1][nt][1]);
                    }
                }
            }
            const uint32_t kp = at + 2 * kT4Keys * C::CODES;
#pragma unroll
            for (int gi = 0; gi < G; ++gi) {
                const float2 s0 = Pair<T>::unpack(lds32(kp + k0 * C::PARAMS + 4 * gi)), s1 = Pair<T>::unpack(lds32(kp + k1 * C::PARAMS + 4 * gi));
                const float m0 = fmaf(8.0f, s0.x, s0.y), m1 = fmaf(8.0f, s1.x, s1.y);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float s = fmaf(e < 2 ? s0.x : s1.x, acc[gi][nt][e], (e < 2 ? m0 : m1) * qsum[gi][nt][e & 1]);
                        z[mt][nt][e] = gi ? z[mt][nt][e] + s : s;
                    }
            }
        }
        if (p.score.cap_out != 0.0f) {                     // cap tanh(x / cap), tanh(x) = 1 - 2 / (1 + e^2x)
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        z[mt][nt][e] = p.score.cap_out * (1.0f - __fdividef(2.0f, 1.0f + exp2f(z[mt][nt][e] * p.score.cap_in)));
        } else {
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[mt][nt][e] *= p.score.sl2;
        }
        uint32_t hidden = 0u;                              // bit 4 (2 mt + e / 2) + 2 nt + e % 2: the query does not see the key
        if (!full) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = chunk * kT4Keys + 8 * i + kappa;
                const bool real = j < n && (there >> i & 1u);
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

        // values' scales: with 2^k the largest power of two in a key's scales, p s = 2^(score + k - M) (s / 2^k), so that
        // what is rounded to T for the second product is at most 2 whatever the values' size
        const uint32_t vp = at + 2 * kT4Keys * C::CODES + kT4Keys * C::PARAMS;
        float2 sm[4][G];
        float inv[4], top[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) top[nt][0] = top[nt][1] = -INFINITY;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float largest = 0.0f;
#pragma unroll
            for (int gi = 0; gi < G; ++gi) {
                sm[i][gi] = Pair<T>::unpack(lds32(vp + (8 * i + kappa) * C::PARAMS + 4 * gi));
                largest = fmaxf(largest, sm[i][gi].x);
            }
            const int k = min(max((int)(__float_as_uint(largest) >> 23) - 127, -24), 60);
            inv[i] = __uint_as_float((uint32_t)(127 - k) << 23);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float& x = z[i >> 1][nt][2 * (i & 1) + e];
                    x += (float)k;
                    top[nt][e] = fmaxf(top[nt][e], x);
                }
        }
        float base[NT][2];
        bool grew = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int s = 4; s < 32; s <<= 1) top[nt][e] = fmaxf(top[nt][e], __shfl_xor_sync(0xffffffffu, top[nt][e], s));
                grew |= top[nt][e] > m[nt][e];
            }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float next = fmaxf(m[nt][e], top[nt][e]);
                    const float f = next == -INFINITY ? 1.0f : exp2_fast(m[nt][e] - next);
                    m[nt][e] = next;
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
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) base[nt][e] = m[nt][e] == -INFINITY ? 0.0f : m[nt][e];

        uint32_t pf[G][2][NT][2];                          // p s / 2^k, the second product's second operand
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float ratio[G], centre[G];
#pragma unroll
            for (int gi = 0; gi < G; ++gi) {
                ratio[gi] = sm[i][gi].x * inv[i];
                centre[gi] = fmaf(8.0f, sm[i][gi].x, sm[i][gi].y) * inv[i];
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float e2[2], w[G][2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    e2[e] = exp2_fast(z[i >> 1][nt][2 * (i & 1) + e] - base[nt][e]);
                    l[nt][e] = fmaf(e2[e], inv[i], l[nt][e]);
                    const bool out = !full && (hidden >> (4 * i + 2 * nt + e) & 1u);       // whatever its scale holds
#pragma unroll
                    for (int gi = 0; gi < G; ++gi) {
                        w[gi][e] = out ? 0.0f : e2[e] * ratio[gi];
                        mid[gi][nt][e] = out ? mid[gi][nt][e] : fmaf(e2[e], centre[gi], mid[gi][nt][e]);
                    }
                }
#pragma unroll
                for (int gi = 0; gi < G; ++gi) pf[gi][i >> 1][nt][i & 1] = transpose8(Pair<T>::pack(w[gi][0], w[gi][1]));
            }
        }

        // O^T += codes^T p: rows are dimensions 64 gi + 8 g + 2 i (c0, c1) and the next one (c2, c3)
        const uint32_t vc = at + kT4Keys * C::CODES;
#pragma unroll
        for (int gi = 0; gi < G; ++gi)
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                uint32_t v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = lds32(vc + code_at<D>(16 * mt + 4 * i + t, 2 * gi + (g >> 2)) + 4 * (g & 3));
                const uint32_t a_lo = __byte_perm(v[0], v[1], 0x5410), a_hi = __byte_perm(v[0], v[1], 0x7632);
                const uint32_t b_lo = __byte_perm(v[2], v[3], 0x5410), b_hi = __byte_perm(v[2], v[3], 0x7632);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint32_t p0 = pf[gi][mt][nt][0], p1 = pf[gi][mt][nt][1];
                    mma_16x8x16<T>(o[gi][0][nt], codes_of<T, 0>(a_lo), codes_of<T, 1>(a_lo), codes_of<T, 0>(b_lo), codes_of<T, 1>(b_lo), p0, p1);
                    mma_16x8x16<T>(o[gi][1][nt], codes_of<T, 2>(a_lo), codes_of<T, 3>(a_lo), codes_of<T, 2>(b_lo), codes_of<T, 3>(b_lo), p0, p1);
                    mma_16x8x16<T>(o[gi][2][nt], codes_of<T, 0>(a_hi), codes_of<T, 1>(a_hi), codes_of<T, 0>(b_hi), codes_of<T, 1>(b_hi), p0, p1);
                    mma_16x8x16<T>(o[gi][3][nt], codes_of<T, 2>(a_hi), codes_of<T, 3>(a_hi), codes_of<T, 2>(b_hi), codes_of<T, 3>(b_hi), p0, p1);
                }
            }

        // the next copy takes the stage that was read in the last turn
        __syncwarp();
        const int ahead = chunk + (kT4Stages - 1) * step, to = stage == 0 ? kT4Stages - 1 : stage - 1;
        if (ahead < chunks) copy(ahead, to, pages[kT4Stages - 1], page_rows[kT4Stages - 1]);
        copies_commit();
#pragma unroll
        for (int i = 0; i < kT4Stages - 1; ++i) {
            pages[i] = pages[i + 1];
            page_rows[i] = page_rows[i + 1];
        }
        look_up(chunk + kT4Stages * step, pages[kT4Stages - 1], page_rows[kT4Stages - 1]);
        stage = stage == kT4Stages - 1 ? 0 : stage + 1;
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
                to[0] = l[nt][e] == 0.0f ? -INFINITY : (m[nt][e] == -INFINITY ? 0.0f : m[nt][e]);
                to[1] = l[nt][e];
            }
#pragma unroll
            for (int gi = 0; gi < G; ++gi) {
                const float back = mid[gi][nt][e];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<float2*>(to + 2 + 64 * gi + 8 * g + 2 * i) = make_float2(o[gi][i][nt][e] + back, o[gi][i][nt][2 + e] + back);
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
        if ((e = cudaFuncSetAttribute(gsr_tree4_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::RING)) != cudaSuccess) return e;
        if (dev <= 63) done.fetch_or(1ull << dev, std::memory_order_release);
    }
    Tree4Plan plan{Divider((uint32_t)p.page), (p.max_nodes * p.group + C::ROWS - 1) / C::ROWS, 1};
    const long long items = (long long)p.B * p.Hkv * plan.tiles;
    const long long chunks = ((long long)p.table_width * p.page + kT4Keys - 1) / kT4Keys;
    while (plan.cluster < 8 && items * plan.cluster < 4ll * sms && chunks > (long long)plan.cluster * kT4Warps) plan.cluster *= 2;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)plan.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(items * plan.cluster));
    cfg.blockDim = dim3(kT4Threads);
    cfg.dynamicSmemBytes = C::RING;
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
