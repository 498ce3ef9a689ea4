// attention_masked_bwd.cuh - gradients of attention with a document or prefix mask, capped scores,
// a distance bias and grouped heads.  Instantiated per element type.
//
// With P_ij = exp(y_ij - lse_i) from the forward pass's log-sum-exp and delta_i = dO_i . O_i,
//     dV_j = sum_i P_ij dO_i
//     dS_ij = P_ij (dO_i . V_j - delta_i) c_ij          c = 1 - tanh^2 with a cap, else 1
//     dQ_i = scale sum_j dS_ij K_j        dK_j = scale sum_i dS_ij Q_i
// dK and dV of a key/value head sum over the query heads of its group.
//
// Three launches: one pass over the rows (delta), then dK and dV by the CTA that owns the keys and
// dQ by the CTA that owns the queries (one more where dK and dV are cut into parts).  The two
// recompute S and dP, seven products of 128 x 128 x D instead of the five that one pass with atomically
// added dQ would take; in return no result depends on the order of atomics, dQ needs no fp32 buffer,
// and every accumulator stays in TMEM from the first product to the last.  dQ's CTAs start on the SMs that
// run out of dK and dV items.  4 x 32 x 4096 x 128 without a mask, bf16: 2850 us, 965 TFLOP/s of the five
// products, 1350 of the seven (68 % of the measured peak); causal 1591 and 864.
//
// fp16: P is carried as 2^12 P and dS as 2^(12 + e) dS, so that neither goes subnormal where a row has many
// keys or dO is small.  |dO_i . V_j - delta_i| <= 2 |dO_i| max|V| (Cauchy-Schwarz; O is a mean of V rows), and e is
// the largest power that keeps dS below 2^15 by this bound: one for each query in dQ, and in dK one for each key,
// for the largest dO_i of the queries that see keys of its document, so that documents and heads with small dO keep
// their digits beside those with large ones.  Either leaves with its row of the accumulator.  max|V| is the
// key/value head's.  bf16 has fp32's range and needs neither.
//
// Masked pairs get P = dS = 0 by selection, but a row of dO, Q or K that is not finite turns 0
// times itself into NaN inside a product.  Where a warp masks, its products and the rows' delta tell: a row of
// Q (of K in dQ's kernel) that is not finite has no finite product, and a row of dO no finite delta.  The warp then
// cleans its half of the tiles before they are weighted ("Infinities and NaN behind a mask" in
// attention_common.cuh).
#pragma once

#include <type_traits>

#include "attention_common.cuh"
#include "ptx_attention.cuh"

namespace gsr {

template <class T>
constexpr float kPShift = Elem<T>::bf16 ? 0.0f : 12.0f;      // log2 of P's factor

// log2 of dS's further factor, from the squares of the bound's two norms.  A capped dS is held without its factor 4
// (weights_chunk), which leaves room for two more bits.
template <class T, int MODE>
__device__ __forceinline__ float ds_shift(float dO2, float v2) {
    if (Elem<T>::bf16) return 0.0f;
    const float n = dO2 * v2;
    if (!(n > 0.0f && n < INFINITY)) return 0.0f;
    const float room = kHasCap<MODE> ? 4.0f : 2.0f;                          // 15 - 12 - 1, and the cap's 2
    return fminf(fmaxf(floorf(room - 0.5f * log2f(n)), -100.0f), 100.0f);    // less log2(bound / 2)
}

// The largest of n values from `at` on that are not negative, by one warp.
__device__ __forceinline__ float warp_max(const float* at, int n, int lane) {
    float m = 0.0f;
    for (int i = lane; i < n; i += 32) m = fmaxf(m, __ldcg(at + i));
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
}
// max|V|^2 of a key/value head.
__device__ __forceinline__ float v_norm(const MaskedBwdParams& p, int b, int hk, int lane) {
    const int tiles = (p.mask.Skv + 63) / 64;
    return warp_max(p.v_norms + ((long long)b * p.mask.Hkv + hk) * tiles, tiles, lane);
}
// max|dO_i|^2 over queries [first, end) of heads [h0, h1), this lane's share: rows up to a multiple of 64, tiles, rows.
// Four loads at once: 2 x 6 heads over 3 of 333 rows 28.9 us so, 30.8 one after another; 2 x 32 over 8 of 567 captured
// 58.3, and 61.0 with eight, whose code is read cold once an item.
__device__ __forceinline__ float dO_norm(const MaskedBwdParams& p, int b, int h0, int h1, int first, int end, int lane) {
    const int up = min((first + 63) / 64 * 64, end), down = max(end / 64 * 64, up);
    const int rows = up - first, tiles = (down - up) / 64, per = rows + tiles + end - down, all = per * (h1 - h0);
    const long long head0 = (long long)b * p.mask.Hq + h0;
    float m = 0.0f;
    for (int i0 = lane; i0 < all; i0 += 4 * 32) {
        float x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * 32, h = i / per, k = i - h * per;
            const bool tile = k >= rows && k < rows + tiles;
            const float* at = tile ? p.tile_norms + (head0 + h) * (p.Sp / 64) + up / 64 + k - rows
                                   : p.row_norms + (head0 + h) * p.Sp + (k < rows ? first + k : down + k - rows - tiles);
            x[u] = i < all ? __ldcg(at) : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) m = fmaxf(m, x[u]);
    }
    return m;
}
// ds_shift of each lane's key, which queries [first, end) see, in steps of heads [h0, h1): the norm is the largest among
// the queries that see one of the warp's keys of the lane's document.  Keys of a document have one end, and the
// first of them the first query.
template <class T, int MODE>
__device__ __forceinline__ float key_shift(const MaskedBwdParams& p, int b, int hk, int h0, int h1, int first, int end, int lane) {
    const int tiles = (p.mask.Skv + 63) / 64;
    const float* v = p.v_norms + ((long long)b * p.mask.Hkv + hk) * tiles;
    const float v_first = lane < tiles ? __ldcg(v + lane) : 0.0f;            // on its way meanwhile
    float mine = 0.0f;
    for (uint32_t left = 0xffffffffu; left;) {
        const int lead = __ffs(left) - 1, f = __shfl_sync(0xffffffffu, first, lead), e = __shfl_sync(0xffffffffu, end, lead);
        const uint32_t same = __ballot_sync(0xffffffffu, end == e) & left;
        if (f < e) {
            const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(dO_norm(p, b, h0, h1, f, e, lane)));
            if (same >> lane & 1u) mine = __uint_as_float(m);
        }
        left &= ~same;
    }
    float v2 = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v_first)));
    if (tiles > 32) v2 = fmaxf(v2, warp_max(v + 32, tiles - 32, lane));
    return ds_shift<T, MODE>(mine, v2);
}

// What a row's exponent offset holds beside -lse: P's power of two, and the constant of a capped
// score (weights_chunk).
template <class T>
__device__ __forceinline__ float row_offset(const ScoreArgs& sc) {
    return kPShift<T> + (sc.cap_in != 0.0f ? sc.cap_out : 0.0f);
}

// ---------------------------------------------------------------------------
// Rows: exponent offsets, delta, and the norms that bound dS
// ---------------------------------------------------------------------------
// A warp takes kWarpRows rows of one head, 16 bytes a lane (D / 8 lanes a row), all loads before the
// first sum; bound by the read of dO and O.  Rows padded to Sp first, then (fp16) the value rows.  A CTA's warps
// share one tile of 64 rows.
constexpr int kWarpRows = 8, kNormRows = 8 * kWarpRows;

// Row r's 8 elements of this lane; zero outside [0, rows).
template <class T>
__device__ __forceinline__ uint4 row_piece(const Strided& t, int b, int h, int r, int rows, int piece) {
    if (r >= rows) return make_uint4(0, 0, 0, 0);
    return __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(t.data) + b * t.batch + h * t.head + r * t.row) + piece);
}
template <class T>
__device__ __forceinline__ float dot8(const uint4& a, const uint4& b) {
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 u = Elem<T>::unpack(x[i]), v = Elem<T>::unpack(y[i]);
        s = fmaf(u.x, v.x, fmaf(u.y, v.y, s));
    }
    return s;
}
template <int LANES>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
// Rows' norms count where they are finite.
__device__ __forceinline__ float finite_norm(float n) { return n < INFINITY ? n : 0.0f; }
// The largest norm of a CTA's rows.
__device__ __forceinline__ void store_tile_norm(float* to, float n) {
    __shared__ uint32_t most[8];
    const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(n));
    if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x < 32) {
        const uint32_t all = __reduce_max_sync(0xffffffffu, threadIdx.x < 8 ? most[threadIdx.x] : 0u);
        if (threadIdx.x == 0) *to = __uint_as_float(all);
    }
}

template <class T, int D>
__global__ void __launch_bounds__(256) gsr_masked_bwd_rows_kernel(const __grid_constant__ MaskedBwdParams p) {
    constexpr int LANES = D / 8, AT_ONCE = 32 / LANES, N = kWarpRows / AT_ONCE;
    const int lane = threadIdx.x & 31, sub = lane / LANES, piece = lane % LANES;
    const MaskArgs& mk = p.mask;
    const int groups = p.Sp / kWarpRows, v_groups = (mk.Skv + kNormRows - 1) / kNormRows * 8;
    long long id = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const long long q_groups = (long long)mk.B * mk.Hq * groups;
    if (id < q_groups) {
        const int bh = (int)(id / groups), i0 = (int)(id - (long long)bh * groups) * kWarpRows, b = bh / mk.Hq, h = bh - b * mk.Hq;
        uint4 x[N], y[N];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            x[n] = row_piece<T>(p.dO, b, h, i0 + n * AT_ONCE + sub, mk.Sq, piece);
            y[n] = row_piece<T>(p.O, b, h, i0 + n * AT_ONCE + sub, mk.Sq, piece);
        }
        // lane r < kWarpRows: row r's interval and lse
        int lo = 0, hi = 0;
        float lse = -INFINITY;
        const int i = i0 + lane;
        if (lane < kWarpRows && i < mk.Sq) {
            row_interval(mk, b, i, lo, hi);
            lse = __ldg(p.lse + ((long long)b * mk.Hq + h) * mk.Sq + i);
        }
        const bool keys = lo < hi && lse != -INFINITY;
        float delta = 0.0f, norm = 0.0f;                 // of row `lane`
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const float d = lanes_sum<LANES>(dot8<T>(x[n], y[n]));
            const float q = Elem<T>::bf16 ? 0.0f : lanes_sum<LANES>(dot8<T>(x[n], x[n]));
#pragma unroll
            for (int k = 0; k < AT_ONCE; ++k) {
                const float dk = __shfl_sync(0xffffffffu, d, k * LANES), qk = __shfl_sync(0xffffffffu, q, k * LANES);
                if (lane == n * AT_ONCE + k) {
                    delta = dk;
                    norm = qk;
                }
            }
        }
        if (lane < kWarpRows) {
            const long long row = (long long)bh * p.Sp + i;
            p.offset[row] = keys ? row_offset<T>(p.score) - lse * kLog2e : -INFINITY;
            // where dO is not finite delta is not either, and says so of a row without keys too (dK's and dV's CTAs look)
            p.neg_delta[row] = keys || !(fabsf(delta) < INFINITY) ? -delta : 0.0f;
        }
        if (!Elem<T>::bf16) {
            norm = keys ? finite_norm(norm) : 0.0f;
            if (lane < kWarpRows) p.row_norms[(long long)bh * p.Sp + i] = norm;
            store_tile_norm(p.tile_norms + id / 8, norm);
        }
        return;
    }
    id -= q_groups;
    if (!Elem<T>::bf16 && id < (long long)mk.B * mk.Hkv * v_groups) {
        const int bh = (int)(id / v_groups), j0 = (int)(id - (long long)bh * v_groups) * kWarpRows, b = bh / mk.Hkv, h = bh - b * mk.Hkv;
        uint4 x[N];
#pragma unroll
        for (int n = 0; n < N; ++n) x[n] = row_piece<T>(p.V, b, h, j0 + n * AT_ONCE + sub, mk.Skv, piece);
        float most = 0.0f;
        bool seen = true;                                // row j0 + lane: padding does not count
        if (mk.num_docs > 0 && lane < kWarpRows) {
            int first = 0, end = 0;
            if (j0 + lane < mk.Skv) key_interval(mk, b, j0 + lane, first, end);
            seen = first < end;
        }
        const unsigned rows_seen = __ballot_sync(0xffffffffu, seen);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const float q = lanes_sum<LANES>(dot8<T>(x[n], x[n]));
            if (rows_seen >> (n * AT_ONCE + sub) & 1u) most = fmaxf(most, finite_norm(q));
        }
        store_tile_norm(p.v_norms + id / 8, most);
    }
}

// Zero rows of a strided output (no queries, or no keys).  One warp per row.
template <class T, int D>
__global__ void __launch_bounds__(256) gsr_masked_zero_kernel(Strided t, int heads, int rows, long long total) {
    const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= total) return;
    const float zero[D / 32] = {};
    const int i = (int)(row % rows), bh = (int)(row / rows);
    store_row<T, D>(static_cast<T*>(t.data) + (bh / heads) * t.batch + (bh % heads) * t.head + i * t.row, threadIdx.x & 31, zero);
}

// ---------------------------------------------------------------------------
// Shared by the two tensor-core kernels
// ---------------------------------------------------------------------------
// 384 threads: warp 0 copies, one lane of warp 1 issues the products, warps 4-11 do the arithmetic
// between them.  Warps w and w + 4 share 32 TMEM lanes and take 64 of the 128 columns each.  The
// threads start with 168 registers each and the first four warps give some to the others: 72 + 2 x
// 216 = 3 x 168.
constexpr int kBwdThreads = 384;
constexpr int kBwdMathWarps = 8;
constexpr int kBwdControlRegs = 72, kBwdMathRegs = 216;
constexpr int kTile = 128;
constexpr int kChunkBytes = 128 * 128;

// 32 raw products -> in place W = 2^x c, where x is the score plus the row's offset less the part of
// it that row_offset holds, and c a quarter of the cap's derivative (r (1 - r); the factor 4 is
// applied with the accumulator's).  `off` gives the offsets of columns i and i + 1; `packed`, where
// wanted, gets 2^x alone in pairs.  `base` as in score_chunk.
template <class T, int MODE, bool PACK, class Off>
__device__ __forceinline__ void weights_chunk(uint32_t (&rr)[32], const ScoreArgs& sc, float slope2, float base, Off off,
                                              uint32_t (&packed)[16]) {
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
        float y0 = __uint_as_float(rr[i]), y1 = __uint_as_float(rr[i + 1]), c0, c1;
        const float2 o = off(i);
        if (kHasCap<MODE>) {
            cap_r_pair(y0, y1, sc.cap_in);
            ffma2(c0, c1, y0, y1, -y0, -y1, y0, y1);
            ffma2(y0, y1, y0, y1, -2.0f * sc.cap_out, -2.0f * sc.cap_out, o.x, o.y);
        } else {
            ffma2(y0, y1, y0, y1, sc.sl2, sc.sl2, o.x, o.y);
        }
        if (kHasBias<MODE>) {
            y0 = fmaf(-slope2, fabsf(base - (float)i), y0);
            y1 = fmaf(-slope2, fabsf(base - (float)(i + 1)), y1);
        }
        y0 = ex2_approx(y0);
        y1 = ex2_approx(y1);
        if (PACK) packed[i / 2] = Elem<T>::pack(y0, y1);
        if (kHasCap<MODE>) fmul2(y0, y1, y0, y1, c0, c1);
        rr[i] = __float_as_uint(y0);
        rr[i + 1] = __float_as_uint(y1);
    }
}
// Whether one of a warp's 32 x 64 products, or of the 64 values at `more` (if any), is not finite.
__device__ __forceinline__ bool products_not_finite(const uint32_t (&a)[32], const uint32_t (&b)[32], const float* more, int lane) {
    float z0 = 0.0f, z1 = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
        ffma2(z0, z1, __uint_as_float(a[i]), __uint_as_float(a[i + 1]), 0.0f, 0.0f, z0, z1);
        ffma2(z0, z1, __uint_as_float(b[i]), __uint_as_float(b[i + 1]), 0.0f, 0.0f, z0, z1);
    }
    if (more) {
        const float2 v = *(reinterpret_cast<const float2*>(more) + lane);
        ffma2(z0, z1, v.x, v.y, 0.0f, 0.0f, z0, z1);
    }
    return __any_sync(0xffffffffu, z0 + z1 != 0.0f);
}
// 64 rows of a tile's chunks in shared memory without what is not finite; true if there was something.  Kept out of
// the kernels' own code (in it, 1 % slower).
template <class T, int DCH>
__device__ __noinline__ bool clean_half_tile(uint8_t* tile, int half, int lane) {
    bool any = false;
#pragma unroll 1
    for (int c = 0; c < DCH; ++c) any |= zero_not_finite<T>(tile + c * kChunkBytes + half * 8192, 512, lane);
    return any;
}
template <int MODE>
constexpr float kCapFactor = kHasCap<MODE> ? 4.0f : 1.0f;

// ---------------------------------------------------------------------------
// dK and dV
// ---------------------------------------------------------------------------
// A work item is 128 keys of one key/value head; its steps are the query tiles that see any of them,
// for every query head of the group.  Where such items are few for the SMs (few key/value heads, one
// batch row), their steps are cut into p.splits equal runs, each an item that leaves its sums in
// fp32 in the workspace, and another launch adds them up in order.  Per step
//     S^T = K Q^T,  dP^T = V dO^T       [128 keys x 128 queries] into 128 TMEM columns each
//     P^T over S^T's columns, dV += P^T dO;   dS^T over dP^T's columns, dK += dS^T Q
// with P^T and dS^T read from TMEM.  At D = 128 the four fill all 512 columns.  The products are
// issued in the order S(n), dK(n-1), dP(n), dV(n): each finds its operand ready because the
// arithmetic of the step before it runs meanwhile, and a region is overwritten only after the
// product that reads it (one thread's products complete in order).  Q is read by S(n) and, a step
// later, by dK(n), so its ring has three entries where dO's has two.
template <class T_, int D_, int MODE_>
struct DkvCfg {
    using T = T_;
    static constexpr int D = D_, MODE = MODE_;
    static constexpr int DCH = D / 64;
    static constexpr int TILE_BYTES = kTile * D * 2;
    static constexpr int NQ = 3, NO = 2;              // ring entries of Q and of dO (with the rows' values)
    static constexpr int OFF_K = 0;
    static constexpr int OFF_V = OFF_K + TILE_BYTES;
    static constexpr int OFF_Q = OFF_V + TILE_BYTES;
    static constexpr int OFF_O = OFF_Q + NQ * TILE_BYTES;
    static constexpr int OFF_ROWS = OFF_O + NO * TILE_BYTES;    // per entry: 128 offsets, 128 -delta
    static constexpr int OFF_BAR = OFF_ROWS + NO * 1024;
    static constexpr int NUM_BARS = 26;
    static constexpr int OFF_CLC = OFF_BAR + NUM_BARS * 8;
    static constexpr int OFF_ITEM = OFF_CLC + 16;
    static constexpr int OFF_CLEANED = OFF_ITEM + 64;           // 4 words
    static constexpr int OFF_MISC = OFF_CLEANED + 16;
    static constexpr int SMEM_BYTES = OFF_MISC + 16;
    static constexpr uint32_t T_S = 0, T_DP = 128, T_DV = 256, T_DK = 256 + D;
    static constexpr uint32_t IDESC_S = idesc_16_f32(Elem<T>::bf16, kTile, kTile, false, false);
    static constexpr uint32_t IDESC_ACC = idesc_16_f32(Elem<T>::bf16, kTile, D, false, true);
    static_assert(SMEM_BYTES <= 232448 && OFF_CLC % 16 == 0, "shared memory");
};

// Products of a 128 x D by a 128 x D operand, both K-major: 128 x 128 into `d`.
template <int D>
__device__ __forceinline__ void mma_tiles(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
        const uint32_t off = (k >> 2) * kChunkBytes + (k & 3) * 32;
        mma_f16_ss(d, smem_desc_sw128(a + off, 16, 1024), smem_desc_sw128(b + off, 16, 1024), idesc, k > 0 ? 1u : 0u);
    }
}

// d (+)= A B with A 128 x 128 in TMEM, its k columns 0-63 packed from `a` on and 64-127 from
// a + 64 on (each half overlays the fp32 columns of the warps that wrote it), and B's rows (k) at `b`.
__device__ __forceinline__ void mma_overlay(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate) {
#pragma unroll
    for (int k = 0; k < kTile / 16; ++k)
        mma_f16_ts(d, a + (k >> 2) * 64 + (k & 3) * 8, smem_desc_sw128(b + k * 2048, kChunkBytes, 1024), idesc,
                   (accumulate || k > 0) ? 1u : 0u);
}

// Rows of an accumulator to a strided output, one row per thread.
template <class T, int D>
__device__ __forceinline__ void store_accumulator(uint32_t col, float factor, bool zero, bool write, T* row) {
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {                   // one copy of the code: it runs cold, once an item
        uint32_t rr[32];
        __syncwarp();                                    // whole warps at the TMEM accesses
        tmem_ld_32x32b_x32(col + c * 32, rr);
        tmem_ld_wait(rr);
        if (zero) {
#pragma unroll
            for (int i = 0; i < 32; ++i) rr[i] = 0u;
        }
        if (write) {
            uint32_t v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float a = __uint_as_float(rr[2 * i]), b = __uint_as_float(rr[2 * i + 1]);
                v[i] = Elem<T>::pack(a * factor, b * factor);
            }
            store_64_bytes(row + c * 32, v);
        }
    }
}

// Row j of part `split` of dV (which 0) or dK (1) in the workspace.
__device__ __forceinline__ float* part_row(const MaskedBwdParams& p, int which, int split, int bh, int j, int D) {
    return p.parts + ((((long long)which * p.splits + split) * (p.mask.B * p.mask.Hkv) + bh) * p.mask.Skv + j) * D;
}

// A warp's rows of dV or dK (`which` 0 or 1), of a whole item or of part `split`, are written, and edge tiles were cleaned:
// what their rows mean to the keys that their queries see.  Steps [begin, end) as in the kernel's Item.  dS of
// a pair whose Q is not finite is NaN or 0, so dK's column is NaN; P is not negative.
template <class T, int D>
__device__ __noinline__ void spread_dkv(const MaskedBwdParams& p, int which, int b, int hk, int k0, int t0, int t1, int begin, int end,
                                        int split) {
    const MaskArgs& mk = p.mask;
    const int lane = threadIdx.x & 31, j = k0 + (threadIdx.x >> 5 & 3) * 32 + lane;
    int all_first, all_end, none, lo = 0, hi = 0;        // the queries that see all keys of the tile
    key_interval(mk, b, k0, none, all_end);
    key_interval(mk, b, min(k0 + kTile, mk.Skv) - 1, all_first, none);
    if (j < mk.Skv) key_interval(mk, b, j, lo, hi);
    for (int k = begin; k < end; ++k) {
        const int t = t0 + k % (t1 - t0), h = hk * mk.group + k / (t1 - t0), i0 = t * kTile;
        if (i0 >= all_first && i0 + kTile <= all_end) continue;
        const Strided& from = which ? p.Q : p.dO;
        const T* rows = static_cast<const T*>(from.data) + b * from.batch + h * from.head;
        const int i1 = min(i0 + kTile, mk.Sq);
        if (p.splits > 1) {
            float* to = part_row(p, which, split, b * mk.Hkv + hk, j, D);
            if (which)
                spread_not_finite<T, D, true>(rows, from.row, i0, i1, lo, hi, to, j < mk.Skv, lane);
            else
                spread_not_finite<T, D, false>(rows, from.row, i0, i1, lo, hi, to, j < mk.Skv, lane);
        } else {
            const Strided& out = which ? p.dK : p.dV;
            uint16_t* to = static_cast<uint16_t*>(out.data) + b * out.batch + hk * out.head + (long long)j * out.row;
            if (which)
                spread_not_finite<T, D, true>(rows, from.row, i0, i1, lo, hi, to, j < mk.Skv, lane);
            else
                spread_not_finite<T, D, false>(rows, from.row, i0, i1, lo, hi, to, j < mk.Skv, lane);
        }
    }
    __syncwarp();
}

// The parts' sums, in order.  A warp takes kSumRows rows of dK or dV, the loads of kSumParts parts before
// their sums; bound by the read of the parts.
constexpr int kSumRows = 2, kSumParts = 4;
template <class T, int D>
__global__ void __launch_bounds__(256) gsr_masked_dkv_sum_kernel(const __grid_constant__ MaskedBwdParams p) {
    using V = typename std::conditional<D == 128, float4, float2>::type;
    const MaskArgs& mk = p.mask;
    const int lane = threadIdx.x & 31;
    const long long rows = (long long)mk.B * mk.Hkv * mk.Skv, first = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * kSumRows;
    grid_wait();                                         // dQ has finished, and dK and dV before it
    float sum[kSumRows][D / 32] = {};
    for (int s0 = 0; s0 < p.splits; s0 += kSumParts) {
        V x[kSumRows][kSumParts];
#pragma unroll
        for (int k = 0; k < kSumRows; ++k)
#pragma unroll
            for (int s = 0; s < kSumParts; ++s) {
                // dV's parts lie before dK's; behind the last part or row a load of it, so that none is conditional
                const long long id = min(first + k, 2 * rows - 1), row = id < rows ? id : id - rows;
                const long long part = (id < rows ? 0 : p.splits) + min(s0 + s, p.splits - 1);
                x[k][s] = *(reinterpret_cast<const V*>(p.parts + (part * rows + row) * D) + lane);
            }
#pragma unroll
        for (int k = 0; k < kSumRows; ++k)
#pragma unroll
            for (int s = 0; s < kSumParts; ++s)
#pragma unroll
                for (int e = 0; e < D / 32; ++e) sum[k][e] += s0 + s < p.splits ? reinterpret_cast<const float*>(&x[k][s])[e] : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < kSumRows; ++k) {
        const long long id = first + k;
        if (id >= 2 * rows) return;
        const int which = id >= rows;
        const long long row = id - (which ? rows : 0);
        const int bh = (int)(row / mk.Skv), j = (int)(row - (long long)bh * mk.Skv), b = bh / mk.Hkv, hk = bh - b * mk.Hkv;
        const Strided& out = which ? p.dK : p.dV;
        store_row<T, D>(static_cast<T*>(out.data) + b * out.batch + hk * out.head + (long long)j * out.row, lane, sum[k]);
    }
}

template <class Cfg>
__global__ void __launch_bounds__(kBwdThreads, 1)
    gsr_masked_dkv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                          const __grid_constant__ MaskedBwdParams p) {
    using T = typename Cfg::T;
    constexpr int D = Cfg::D, DCH = Cfg::DCH, NQ = Cfg::NQ, NO = Cfg::NO;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023u) {
        if (threadIdx.x == 0) atomicCAS(p.err, 0, kDevErrKernelMaskedDkv | kDevErrLayout);
        return;
    }
    const uint32_t sb = smem_u32(smem);
    auto bar = [&](int i) { return sb + Cfg::OFF_BAR + 8u * i; };
    auto q_full = [&](int s) { return bar(0 + s); };
    auto q_empty = [&](int s) { return bar(3 + s); };
    auto o_full = [&](int s) { return bar(6 + s); };
    auto o_empty = [&](int s) { return bar(8 + s); };
    auto rows_empty = [&](int s) { return bar(10 + s); };
    auto item_pub = [&](int i) { return bar(12 + i); };
    auto item_read = [&](int i) { return bar(14 + i); };
    const uint32_t kv_full = bar(16), kv_empty = bar(17), s_full = bar(18), p_full = bar(19), dp_full = bar(20),
                   ds_full = bar(21), done = bar(22), clc = bar(23), drain = bar(24);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::OFF_MISC);
    volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + Cfg::OFF_MISC + 4);
    volatile int* item_box = reinterpret_cast<volatile int*>(smem + Cfg::OFF_ITEM);
    // cleaned[n & 3] == n: a tile of item n was cleaned.  (Item n + 4 is published once every warp is past n.)
    volatile uint32_t* cleaned = reinterpret_cast<volatile uint32_t*>(smem + Cfg::OFF_CLEANED);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const MaskArgs& mk = p.mask;

    // What the producer publishes; b < 0: no more items.  Query tiles [t0, t1) see some of the keys;
    // step k is tile t0 + k % (t1 - t0) of the group's head k / (t1 - t0), and the item runs steps
    // [begin, end) of them, as part `split` of p.splits.
    struct Item {
        int b, hk, k0, t0, t1, begin, end, split;
    };
    auto read_item = [&](int box) {
        volatile int* v = item_box + 8 * box;
        return Item{v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]};
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < NQ; ++s) {
            mbar_init(q_full(s), 1);
            mbar_init(q_empty(s), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(o_full(s), 1);
            mbar_init(o_empty(s), 1);
            mbar_init(rows_empty(s), 1);
            mbar_init(item_pub(s), 1);
            mbar_init(item_read(s), 1 + kBwdMathWarps);
        }
        mbar_init(kv_full, 1);
        mbar_init(kv_empty, 1);
        mbar_init(s_full, 1);
        mbar_init(p_full, kBwdMathWarps);
        mbar_init(dp_full, 1);
        mbar_init(ds_full, kBwdMathWarps);
        mbar_init(done, 1);
        mbar_init(clc, 1);
        mbar_init(drain, 1);
        for (int i = 0; i < 4; ++i) cleaned[i] = 0u;
        *abort_flag = 0u;
        fence_mbarrier_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
        tma_prefetch_desc(&tmO);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish_alloc_permit();
    }
    grid_wait();                                         // the rows' values
    grid_launch_next();                                  // dQ needs no more than they
    tcgen05_fence_before();
    __syncthreads();
    tcgen05_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const Waiter w{p.err, p.timeout_ns, abort_flag, kDevErrKernelMaskedDkv};

    if (warp < 4) {
        reg_dec<kBwdControlRegs>();
        if (warp == 0) {
            // ------------------------------------------------------------ items + TMA producer
            const uint64_t pol = l2_policy_evict_last();     // Q and dO are read by every key tile
            const int n_kt = (mk.Skv + kTile - 1) / kTile;
            uint32_t n_pub = 0, n_item = 0, n_clc = 0, n = 0;   // items published, items with steps, answers, steps
            uint32_t armed = 0, parity = 0;                  // per barrier q_full 0-2, o_full 3-4, kv_full 5
            bool drop = (p.test_flags & kTestDropFirstLoad) && blockIdx.x == 0;
            bool asked = false;
            int item = blockIdx.x;
            auto arm = [&](int i, uint32_t ph) {
                armed |= 1u << i;
                parity = (parity & ~(1u << i)) | (ph & 1u) << i;
            };
            while (true) {
                Item it{-1, 0, 0, 0, 0, 0, 0, 0};
                if (item >= 0) {
                    // key tiles from the first (under a causal mask the most queries see it) to the last,
                    // in groups of key/value heads whose Q and dO stay in L2 together
                    const int per_group = p.kv_head_group * n_kt * p.splits, grp = item / per_group, r_in = item - grp * per_group;
                    const int gsz = min(mk.B * mk.Hkv - grp * p.kv_head_group, p.kv_head_group);
                    const int bh = grp * p.kv_head_group + r_in % gsz;
                    it.b = bh / mk.Hkv;
                    it.hk = bh - it.b * mk.Hkv;
                    it.split = r_in / gsz % p.splits;
                    it.k0 = r_in / gsz / p.splits * kTile;
                    // lane 0: the queries that see the tile's first key, lane 1: its last
                    int first = 0, end = 0;
                    if (lane < 2) key_interval(mk, it.b, lane == 0 ? it.k0 : min(it.k0 + kTile, mk.Skv) - 1, first, end);
                    end = __shfl_sync(0xffffffffu, end, 1);
                    first = __shfl_sync(0xffffffffu, first, 0);
                    it.t0 = first / kTile;
                    it.t1 = first < end ? (end + kTile - 1) / kTile : it.t0;
                    const long long steps = (long long)(it.t1 - it.t0) * mk.group;
                    it.begin = (int)(steps * it.split / p.splits);
                    it.end = (int)(steps * (it.split + 1) / p.splits);
                }
                const uint32_t box = n_pub & 1u;
                bool ok = lane != 0 || w.wait(item_read(box), ((n_pub >> 1) & 1u) ^ 1u, kDevErrProducerEmpty);
                if (!__all_sync(0xffffffffu, ok)) break;
                if (lane == 0) {
                    volatile int* v = item_box + 8 * box;
                    v[0] = it.b;
                    v[1] = it.hk;
                    v[2] = it.k0;
                    v[3] = it.t0;
                    v[4] = it.t1;
                    v[5] = it.begin;
                    v[6] = it.end;
                    v[7] = it.split;
                    mbar_arrive(item_pub(box));
                }
                ++n_pub;
                if (item < 0) break;
                if (lane == 0) {
                    if (it.begin < it.end) {
                        ok = w.wait(kv_empty, (n_item & 1u) ^ 1u, kDevErrProducerEmpty);
                        if (ok && !drop) {
                            mbar_arrive_expect_tx(kv_full, 2 * Cfg::TILE_BYTES);
#pragma unroll
                            for (int c = 0; c < DCH; ++c) {
                                tma_load_4d(sb + Cfg::OFF_K + c * kChunkBytes, &tmK, kv_full, c * 64, it.k0, it.hk, it.b, pol);
                                tma_load_4d(sb + Cfg::OFF_V + c * kChunkBytes, &tmV, kv_full, c * 64, it.k0, it.hk, it.b, pol);
                            }
                            arm(5, n_item);
                        }
                        drop = false;                        // test hook: the first K and V are never loaded
                        ++n_item;
                        const int tiles = it.t1 - it.t0;
                        for (int k = it.begin; ok && k < it.end; ++k, ++n) {
                            const int h = it.hk * mk.group + k / tiles, t = it.t0 + k % tiles;
                            const long long row0 = ((long long)it.b * mk.Hq + h) * p.Sp;
                            const int sq = (int)(n % NQ), so = (int)(n % NO);
                            const uint32_t ph_q = n / NQ, ph_o = n / NO;
                            if (!(ok = w.wait(q_empty(sq), (ph_q & 1u) ^ 1u, kDevErrProducerEmpty))) break;
                            mbar_arrive_expect_tx(q_full(sq), Cfg::TILE_BYTES);
#pragma unroll
                            for (int c = 0; c < DCH; ++c)
                                tma_load_4d(sb + Cfg::OFF_Q + sq * Cfg::TILE_BYTES + c * kChunkBytes, &tmQ, q_full(sq), c * 64,
                                            t * kTile, h, it.b, pol);
                            arm(sq, ph_q);
                            if (!(ok = w.wait(o_empty(so), (ph_o & 1u) ^ 1u, kDevErrProducerEmpty) &&
                                       w.wait(rows_empty(so), (ph_o & 1u) ^ 1u, kDevErrProducerEmpty)))
                                break;
                            mbar_arrive_expect_tx(o_full(so), Cfg::TILE_BYTES + 1024);
#pragma unroll
                            for (int c = 0; c < DCH; ++c)
                                tma_load_4d(sb + Cfg::OFF_O + so * Cfg::TILE_BYTES + c * kChunkBytes, &tmO, o_full(so), c * 64,
                                            t * kTile, h, it.b, pol);
                            bulk_load(sb + Cfg::OFF_ROWS + so * 1024, p.offset + row0 + t * kTile, 512, o_full(so));
                            bulk_load(sb + Cfg::OFF_ROWS + so * 1024 + 512, p.neg_delta + row0 + t * kTile, 512, o_full(so));
                            arm(3 + so, ph_o);
                        }
                    }
                    // the next item, asked for once this one's copies are issued: earlier, a CTA busy with a
                    // long item would hold one that another could start
                    if (ok) {
                        fence_proxy_async_smem();            // the last answer has been read
                        mbar_arrive_expect_tx(clc, 16);
                        clc_try_cancel(sb + Cfg::OFF_CLC, clc);
                        asked = true;
                        if ((ok = w.wait(clc, n_clc & 1u, kDevErrProducerEmpty))) {
                            asked = false;
                            item = clc_taken(sb + Cfg::OFF_CLC);
                        }
                    }
                }
                ++n_clc;
                if (!__all_sync(0xffffffffu, ok)) break;
                item = __shfl_sync(0xffffffffu, item, 0);
            }
            if (lane == 0) {   // every copy and answer under way must land before the CTA may exit
                if (asked) w.drain(clc, (n_clc - 1) & 1u);
                for (int i = 0; i < 6; ++i)
                    if (armed & (1u << i)) w.drain(i < 3 ? q_full(i) : (i < 5 ? o_full(i - 3) : kv_full), (parity >> i) & 1u);
            }
            __syncwarp();
        } else if (warp == 1) {
            // ------------------------------------------------------------ MMA issuer
            if (lane == 0) {
                uint32_t n_box = 0, n_item = 0, n = 0;
                bool ok = true;
                const uint32_t k_s = sb + Cfg::OFF_K, v_s = sb + Cfg::OFF_V;
                while (ok) {
                    const uint32_t box = n_box & 1u;
                    if (!w.wait(item_pub(box), (n_box >> 1) & 1u, kDevErrMmaFull)) break;
                    const Item it = read_item(box);
                    mbar_arrive(item_read(box));
                    ++n_box;
                    if (it.b < 0) break;
                    const int steps = it.end - it.begin;
                    if (steps <= 0) continue;
                    if (!w.wait(kv_full, n_item & 1u, kDevErrMmaFull)) break;
                    ++n_item;
                    // dK += dS^T(m) Q(m), once dS^T(m) is written; the step's Q and row values are then free
                    auto issue_dk = [&](uint32_t m, bool first) {
                        if (!w.wait(ds_full, m & 1u, kDevErrMmaFull)) return false;
                        tcgen05_fence_after();
                        mma_overlay(tmem_base + Cfg::T_DK, tmem_base + Cfg::T_DP, sb + Cfg::OFF_Q + (m % NQ) * Cfg::TILE_BYTES,
                                    Cfg::IDESC_ACC, !first);
                        mma_commit(q_empty((int)(m % NQ)));
                        mma_commit(rows_empty((int)(m % NO)));
                        return true;
                    };
                    for (int i = 0; i < steps; ++i, ++n) {
                        const int sq = (int)(n % NQ), so = (int)(n % NO);
                        if (!(ok = w.wait(q_full(sq), (n / NQ) & 1u, kDevErrMmaFull))) break;
                        tcgen05_fence_after();
                        mma_tiles<D>(tmem_base + Cfg::T_S, k_s, sb + Cfg::OFF_Q + sq * Cfg::TILE_BYTES, Cfg::IDESC_S);
                        mma_commit(s_full);
                        if (i > 0 && !(ok = issue_dk(n - 1, i == 1))) break;
                        if (!(ok = w.wait(o_full(so), (n / NO) & 1u, kDevErrMmaFull))) break;
                        tcgen05_fence_after();
                        const uint32_t o_s = sb + Cfg::OFF_O + so * Cfg::TILE_BYTES;
                        mma_tiles<D>(tmem_base + Cfg::T_DP, v_s, o_s, Cfg::IDESC_S);
                        mma_commit(dp_full);
                        if (!(ok = w.wait(p_full, n & 1u, kDevErrMmaFull))) break;
                        tcgen05_fence_after();
                        mma_overlay(tmem_base + Cfg::T_DV, tmem_base + Cfg::T_S, o_s, Cfg::IDESC_ACC, i > 0);
                        mma_commit(o_empty(so));
                    }
                    if (!ok || !(ok = issue_dk(n - 1, steps == 1))) break;
                    mma_commit(kv_empty);
                    mma_commit(done);
                }
                mma_commit(drain);
                w.drain(drain, 0);
            }
            __syncwarp();
        }
    } else {
        reg_inc<kBwdMathRegs>();
        // ------------------------------------------------------------ P, dS and the output (warps 4-11)
        const int half = (warp - 4) >> 2;                // query columns 64 half .. + 63
        const int quad = warp & 3;
        const int r = quad * 32 + lane;                  // key of the tile
        const uint32_t lane_base = tmem_base + ((uint32_t)(quad * 32) << 16);
        const uint32_t s_col = lane_base + Cfg::T_S + half * 64, dp_col = lane_base + Cfg::T_DP + half * 64;
        uint32_t n_box = 0, n = 0, n_done = 0;
        bool ok = true;
        while (ok) {
            const uint32_t box = n_box & 1u;
            if (!__all_sync(0xffffffffu, w.wait(item_pub(box), (n_box >> 1) & 1u, kDevErrEpilogueFull))) break;
            const Item it = read_item(box);
            __syncwarp();
            if (lane == 0) mbar_arrive(item_read(box));
            ++n_box;
            if (it.b < 0) break;
            const int j = it.k0 + r;
            int first = 0, end = INT_MAX;                // the queries that see this thread's key (behind the last: no mask)
            if (j < mk.Skv) key_interval(mk, it.b, j, first, end);
            float shift = 0.0f, ds_mul = 1.0f;
            if (!Elem<T>::bf16 && it.begin < it.end) {
                const int h0 = it.hk * mk.group, per = it.t1 - it.t0;
                shift = key_shift<T, Cfg::MODE>(p, it.b, it.hk, h0 + it.begin / per, h0 + (it.end - 1) / per + 1, first,
                                                j < mk.Skv ? end : 0, lane);
                ds_mul = exp2f(shift);
            }
            const int tiles = max(it.t1 - it.t0, 1);
            int h = it.hk * mk.group + it.begin / tiles, t = it.t0 + it.begin % tiles;
            for (int k = it.begin; k < it.end; ++k, ++n, ++t) {
                if (t == it.t1) {
                    t = it.t0;
                    ++h;
                }
                const float slope2 = kHasBias<Cfg::MODE> ? __ldg(p.score.slopes + h) * kLog2e : 0.0f;
                const int i0 = t * kTile + half * 64;
                const bool masked = __any_sync(0xffffffffu, i0 < first || i0 + 64 > end);
                if (!__all_sync(0xffffffffu, w.wait(o_full((int)(n % NO)), (n / NO) & 1u, kDevErrEpilogueFull) &&
                                                 w.wait(s_full, n & 1u, kDevErrEpilogueFull))) {
                    ok = false;
                    break;
                }
                tcgen05_fence_after();
                const float* rows = reinterpret_cast<const float*>(smem + Cfg::OFF_ROWS + (n % NO) * 1024) + half * 64;
                const float base = (float)(j - mk.offset - i0);
                uint32_t w0[32], w1[32];
                tmem_ld_32x32b_x32(s_col, w0);
                tmem_ld_32x32b_x32(s_col + 32, w1);
                tmem_ld_wait(w0);
                reg_tie(w1);
                if (masked && __builtin_expect(products_not_finite(w0, w1, rows + 128, lane), 0)) {
                    // dP takes dO as it is
                    if (!__all_sync(0xffffffffu, w.wait(dp_full, n & 1u, kDevErrEpilogueFull))) {
                        ok = false;
                        break;
                    }
                    if (clean_half_tile<T, DCH>(smem + Cfg::OFF_Q + (n % NQ) * Cfg::TILE_BYTES, half, lane) |
                        clean_half_tile<T, DCH>(smem + Cfg::OFF_O + (n % NO) * Cfg::TILE_BYTES, half, lane))
                        cleaned[n_box & 3u] = n_box;
                    fence_proxy_async_smem();
                    if (kHasCap<Cfg::MODE>) {            // a hidden NaN would take its visible neighbour along
                        const uint32_t v0 = between(first - i0, end - i0), v1 = between(first - i0 - 32, end - i0 - 32);
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            if (!(v0 >> i & 1u)) w0[i] = 0u;
                            if (!(v1 >> i & 1u)) w1[i] = 0u;
                        }
                    }
                }
                auto p_chunk = [&](uint32_t (&rr)[32], int c) {
                    uint32_t packed[16];
                    weights_chunk<T, Cfg::MODE, true>(rr, p.score, slope2, base - (float)(c * 32),
                                                      [&](int i) { return *reinterpret_cast<const float2*>(rows + c * 32 + i); },
                                                      packed);
                    if (masked) {
                        const uint32_t vis = between(first - i0 - c * 32, end - i0 - c * 32);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!(vis >> i & 1u)) {
                                rr[i] = 0u;
                                packed[i / 2] &= i & 1 ? 0x0000ffffu : 0xffff0000u;
                            }
                    }
                    tmem_st_32x32b_x16(s_col + c * 16, packed);
                    if (!Elem<T>::bf16) {
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            float a, b;
                            fmul2(a, b, __uint_as_float(rr[i]), __uint_as_float(rr[i + 1]), ds_mul, ds_mul);
                            rr[i] = __float_as_uint(a);
                            rr[i + 1] = __float_as_uint(b);
                        }
                    }
                };
                p_chunk(w0, 0);
                p_chunk(w1, 1);
                tmem_st_wait();
                tcgen05_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full);
                if (!__all_sync(0xffffffffu, w.wait(dp_full, n & 1u, kDevErrEpilogueFull))) {
                    ok = false;
                    break;
                }
                tcgen05_fence_after();
                uint32_t dp0[32], dp1[32];
                tmem_ld_32x32b_x32(dp_col, dp0);
                tmem_ld_32x32b_x32(dp_col + 32, dp1);
                tmem_ld_wait(dp0);
                reg_tie(dp1);
                auto ds_chunk = [&](const uint32_t (&ww)[32], const uint32_t (&dp)[32], int c) {
                    uint32_t packed[16];
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float2 nd = *reinterpret_cast<const float2*>(rows + 128 + c * 32 + i);
                        float d0 = __uint_as_float(dp[i]), d1 = __uint_as_float(dp[i + 1]);
                        fadd2(d0, d1, nd.x, nd.y);
                        fmul2(d0, d1, d0, d1, __uint_as_float(ww[i]), __uint_as_float(ww[i + 1]));
                        packed[i / 2] = Elem<T>::pack(d0, d1);
                    }
                    if (masked) {
                        const uint32_t vis = between(first - i0 - c * 32, end - i0 - c * 32);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!(vis >> i & 1u)) packed[i / 2] &= i & 1 ? 0x0000ffffu : 0xffff0000u;
                    }
                    tmem_st_32x32b_x16(dp_col + c * 16, packed);
                };
                ds_chunk(w0, dp0, 0);
                ds_chunk(w1, dp1, 1);
                tmem_st_wait();
                tcgen05_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(ds_full);
            }
            if (!ok) break;
            const bool none = it.begin >= it.end;
            if (!none) {
                ok = __all_sync(0xffffffffu, w.wait(done, n_done & 1u, kDevErrEpilogueFull));
                ++n_done;
                tcgen05_fence_after();
                if (!ok) break;
            }
            // half 0 writes dV's rows, half 1 dK's.  The next item's products overwrite the accumulators
            // only after this warp's next P and dS.
            const uint32_t col = lane_base + (half == 0 ? Cfg::T_DV : Cfg::T_DK);
            const float factor = half == 0 ? exp2f(-kPShift<T>) : kCapFactor<Cfg::MODE> * p.score.scale * exp2f(-kPShift<T> - shift);
            if (p.splits > 1) {
                float* row = part_row(p, half, it.split, it.b * mk.Hkv + it.hk, j, D);
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t rr[32];
                    __syncwarp();
                    tmem_ld_32x32b_x32(col + c * 32, rr);
                    tmem_ld_wait(rr);
                    if (j < mk.Skv) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            const float4 v = make_float4(__uint_as_float(rr[i]) * factor, __uint_as_float(rr[i + 1]) * factor,
                                                         __uint_as_float(rr[i + 2]) * factor, __uint_as_float(rr[i + 3]) * factor);
                            *reinterpret_cast<float4*>(row + c * 32 + i) = none ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : v;
                        }
                    }
                }
                tcgen05_fence_before();
            } else {
                const Strided& out = half == 0 ? p.dV : p.dK;
                T* row = static_cast<T*>(out.data) + it.b * out.batch + it.hk * out.head + (long long)j * out.row;
                store_accumulator<T, D>(col, factor, none, j < mk.Skv, row);
                tcgen05_fence_before();
            }
            if (__builtin_expect(cleaned[n_box & 3u] == n_box, 0)) spread_dkv<T, D>(p, half, it.b, it.hk, it.k0, it.t0, it.t1, it.begin, it.end, it.split);
        }
    }

    tcgen05_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tcgen05_fence_after();
        tmem_dealloc(tmem_base, 512);
    }
}

// ---------------------------------------------------------------------------
// dQ
// ---------------------------------------------------------------------------
// A work item is 128 queries of one head; its steps are the key tiles they see.  Per step
//     S = Q K^T,  dP = dO V^T,  dS over dP's columns,  dQ += dS K
// S has one region (the arithmetic takes it into registers at once) and dP two, so that S(n+1) and
// dP(n+1) run on the tensor core while dS(n) is computed; dQ(n) follows.  K is read by S(n) and,
// after that, by dQ(n): three ring entries, two for V.  dS(n+1) may be there before the issuing lane
// looks for dS(n), so the two have a barrier each (on one, its phase would be back where it was).
template <class T_, int D_, int MODE_>
struct DqCfg {
    using T = T_;
    static constexpr int D = D_, MODE = MODE_;
    static constexpr int DCH = D / 64;
    static constexpr int TILE_BYTES = kTile * D * 2;
    static constexpr int NK = 3, NV = 2;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_O = OFF_Q + TILE_BYTES;
    static constexpr int OFF_K = OFF_O + TILE_BYTES;
    static constexpr int OFF_V = OFF_K + NK * TILE_BYTES;
    static constexpr int OFF_BAR = OFF_V + NV * TILE_BYTES;
    static constexpr int NUM_BARS = 26;
    static constexpr int OFF_CLC = OFF_BAR + NUM_BARS * 8;
    static constexpr int OFF_ITEM = OFF_CLC + 16;
    static constexpr int OFF_CLEANED = OFF_ITEM + 64;           // 4 words
    static constexpr int OFF_MISC = OFF_CLEANED + 16;
    static constexpr int SMEM_BYTES = OFF_MISC + 16;
    static constexpr uint32_t T_S = 0, T_DP = 128, T_DQ = 384;
    static constexpr uint32_t IDESC_S = idesc_16_f32(Elem<T>::bf16, kTile, kTile, false, false);
    static constexpr uint32_t IDESC_ACC = idesc_16_f32(Elem<T>::bf16, kTile, D, false, true);
    static_assert(SMEM_BYTES <= 232448 && OFF_CLC % 16 == 0, "shared memory");
};

// A warp's rows of dQ are written, and edge tiles were cleaned: what their keys mean to the rows that see them (NaN, as in dK).
template <class T, int D>
__device__ __noinline__ void spread_dq(const MaskedBwdParams& p, int b, int h, int q_base, int t0, int t1) {
    const MaskArgs& mk = p.mask;
    const int lane = threadIdx.x & 31, qi = q_base + (threadIdx.x >> 5 & 3) * 32 + lane;
    int all_lo, all_hi, none, lo = 0, hi = 0;            // the keys that all rows of the tile see
    row_interval(mk, b, q_base, none, all_hi);
    row_interval(mk, b, min(q_base + kTile, mk.Sq) - 1, all_lo, none);
    if (qi < mk.Sq) row_interval(mk, b, qi, lo, hi);
    const T* rows = static_cast<const T*>(p.K.data) + b * p.K.batch + h / mk.group * p.K.head;
    uint16_t* to = static_cast<uint16_t*>(p.dQ.data) + b * p.dQ.batch + h * p.dQ.head + (long long)qi * p.dQ.row;
    for (int t = t0; t < t1; ++t)
        if (t * kTile < all_lo || (t + 1) * kTile > all_hi)
            spread_not_finite<T, D, true>(rows, p.K.row, t * kTile, min((t + 1) * kTile, mk.Skv), lo, hi, to, qi < mk.Sq, lane);
    __syncwarp();
}

template <class Cfg>
__global__ void __launch_bounds__(kBwdThreads, 1)
    gsr_masked_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                         const __grid_constant__ MaskedBwdParams p) {
    using T = typename Cfg::T;
    constexpr int D = Cfg::D, DCH = Cfg::DCH, NK = Cfg::NK, NV = Cfg::NV;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023u) {
        if (threadIdx.x == 0) atomicCAS(p.err, 0, kDevErrKernelMaskedDq | kDevErrLayout);
        return;
    }
    const uint32_t sb = smem_u32(smem);
    auto bar = [&](int i) { return sb + Cfg::OFF_BAR + 8u * i; };
    auto k_full = [&](int s) { return bar(0 + s); };
    auto k_empty = [&](int s) { return bar(3 + s); };
    auto v_full = [&](int s) { return bar(6 + s); };
    auto v_empty = [&](int s) { return bar(8 + s); };
    auto dp_full = [&](int s) { return bar(10 + s); };
    auto item_pub = [&](int i) { return bar(12 + i); };
    auto item_read = [&](int i) { return bar(14 + i); };
    auto ds_full = [&](int s) { return bar(16 + s); };
    const uint32_t q_full = bar(18), q_empty = bar(19), s_full = bar(20), s_read = bar(21), done = bar(22), clc = bar(23),
                   drain = bar(24);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::OFF_MISC);
    volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + Cfg::OFF_MISC + 4);
    volatile int* item_box = reinterpret_cast<volatile int*>(smem + Cfg::OFF_ITEM);
    // cleaned[n & 3] == n: a tile of item n was cleaned.  (Item n + 4 is published once every warp is past n.)
    volatile uint32_t* cleaned = reinterpret_cast<volatile uint32_t*>(smem + Cfg::OFF_CLEANED);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const MaskArgs& mk = p.mask;

    struct Item {
        int b, h, q_base, t0, t1;
    };
    auto read_item = [&](int box) {
        volatile int* v = item_box + 8 * box;
        return Item{v[0], v[1], v[2], v[3], v[4]};
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < NK; ++s) {
            mbar_init(k_full(s), 1);
            mbar_init(k_empty(s), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(v_full(s), 1);
            mbar_init(v_empty(s), 1);
            mbar_init(dp_full(s), 1);
            mbar_init(ds_full(s), kBwdMathWarps);
            mbar_init(item_pub(s), 1);
            mbar_init(item_read(s), 1 + kBwdMathWarps);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(s_full, 1);
        mbar_init(s_read, kBwdMathWarps);
        mbar_init(done, 1);
        mbar_init(clc, 1);
        mbar_init(drain, 1);
        for (int i = 0; i < 4; ++i) cleaned[i] = 0u;
        *abort_flag = 0u;
        fence_mbarrier_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
        tma_prefetch_desc(&tmO);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish_alloc_permit();
    }
    tcgen05_fence_before();
    __syncthreads();
    tcgen05_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const Waiter w{p.err, p.timeout_ns, abort_flag, kDevErrKernelMaskedDq};

    if (warp < 4) {
        reg_dec<kBwdControlRegs>();
        if (warp == 0) {
            // ------------------------------------------------------------ items + TMA producer
            if (lane == 0) {
                const uint64_t pol = l2_policy_evict_last();
                const int n_qb = (mk.Sq + kTile - 1) / kTile;
                uint32_t n_pub = 0, n_item = 0, n_clc = 0, n = 0;
                uint32_t armed = 0, parity = 0;              // k_full 0-2, v_full 3-4, q_full 5
                bool drop = (p.test_flags & kTestDropFirstLoad) && blockIdx.x == 0;
                bool asked = false, ok = true;
                int item = blockIdx.x;
                auto arm = [&](int i, uint32_t ph) {
                    armed |= 1u << i;
                    parity = (parity & ~(1u << i)) | (ph & 1u) << i;
                };
                while (ok) {
                    Item it{-1, 0, 0, 0, 0};
                    if (item >= 0) {
                        const int per_group = p.q_head_group * n_qb, grp = item / per_group, r_in = item - grp * per_group;
                        const int gsz = min(mk.B * mk.Hq - grp * p.q_head_group, p.q_head_group);
                        const int bh = grp * p.q_head_group + r_in % gsz;
                        it.b = bh / mk.Hq;
                        it.h = bh - it.b * mk.Hq;
                        it.q_base = (n_qb - 1 - r_in / gsz) * kTile;
                        int lo, hi, none;
                        row_interval(mk, it.b, it.q_base, lo, none);
                        row_interval(mk, it.b, min(it.q_base + kTile, mk.Sq) - 1, none, hi);
                        it.t0 = lo / kTile;
                        it.t1 = hi > lo ? (hi + kTile - 1) / kTile : it.t0;
                    }
                    const uint32_t box = n_pub & 1u;
                    if (!(ok = w.wait(item_read(box), ((n_pub >> 1) & 1u) ^ 1u, kDevErrProducerEmpty))) break;
                    volatile int* v = item_box + 8 * box;
                    v[0] = it.b;
                    v[1] = it.h;
                    v[2] = it.q_base;
                    v[3] = it.t0;
                    v[4] = it.t1;
                    mbar_arrive(item_pub(box));
                    ++n_pub;
                    if (item < 0) break;
                    if (it.t0 < it.t1) {
                        if (!(ok = w.wait(q_empty, (n_item & 1u) ^ 1u, kDevErrProducerEmpty))) break;
                        if (!drop) {
                            mbar_arrive_expect_tx(q_full, 2 * Cfg::TILE_BYTES);
#pragma unroll
                            for (int c = 0; c < DCH; ++c) {
                                tma_load_4d(sb + Cfg::OFF_Q + c * kChunkBytes, &tmQ, q_full, c * 64, it.q_base, it.h, it.b, pol);
                                tma_load_4d(sb + Cfg::OFF_O + c * kChunkBytes, &tmO, q_full, c * 64, it.q_base, it.h, it.b, pol);
                            }
                            arm(5, n_item);
                        }
                        drop = false;                        // test hook: the first Q and dO are never loaded
                        ++n_item;
                        const int hk = it.h / mk.group;
                        for (int t = it.t0; t < it.t1; ++t, ++n) {
                            const int sk = (int)(n % NK), sv = (int)(n % NV);
                            if (!(ok = w.wait(k_empty(sk), ((n / NK) & 1u) ^ 1u, kDevErrProducerEmpty))) break;
                            mbar_arrive_expect_tx(k_full(sk), Cfg::TILE_BYTES);
#pragma unroll
                            for (int c = 0; c < DCH; ++c)
                                tma_load_4d(sb + Cfg::OFF_K + sk * Cfg::TILE_BYTES + c * kChunkBytes, &tmK, k_full(sk), c * 64, t * kTile,
                                            hk, it.b, pol);
                            arm(sk, n / NK);
                            if (!(ok = w.wait(v_empty(sv), ((n / NV) & 1u) ^ 1u, kDevErrProducerEmpty))) break;
                            mbar_arrive_expect_tx(v_full(sv), Cfg::TILE_BYTES);
#pragma unroll
                            for (int c = 0; c < DCH; ++c)
                                tma_load_4d(sb + Cfg::OFF_V + sv * Cfg::TILE_BYTES + c * kChunkBytes, &tmV, v_full(sv), c * 64, t * kTile,
                                            hk, it.b, pol);
                            arm(3 + sv, n / NV);
                        }
                        if (!ok) break;
                    }
                    fence_proxy_async_smem();                // the last answer has been read
                    mbar_arrive_expect_tx(clc, 16);
                    clc_try_cancel(sb + Cfg::OFF_CLC, clc);
                    asked = true;
                    ++n_clc;
                    if (!(ok = w.wait(clc, (n_clc - 1) & 1u, kDevErrProducerEmpty))) break;
                    asked = false;
                    item = clc_taken(sb + Cfg::OFF_CLC);
                }
                if (asked) w.drain(clc, (n_clc - 1) & 1u);
                for (int i = 0; i < 6; ++i)
                    if (armed & (1u << i)) w.drain(i < 3 ? k_full(i) : (i < 5 ? v_full(i - 3) : q_full), (parity >> i) & 1u);
            }
            __syncwarp();
        } else if (warp == 1) {
            // ------------------------------------------------------------ MMA issuer
            if (lane == 0) {
                uint32_t n_box = 0, n_item = 0, n = 0;
                bool ok = true;
                const uint32_t q_s = sb + Cfg::OFF_Q, o_s = sb + Cfg::OFF_O;
                // S(m) and dP(m), once their operands have landed and S(m-1) is in registers
                auto issue_scores = [&](uint32_t m, bool first) {
                    if (!w.wait(k_full((int)(m % NK)), (m / NK) & 1u, kDevErrMmaFull)) return false;
                    if (!first && !w.wait(s_read, (m - 1) & 1u, kDevErrMmaFull)) return false;
                    tcgen05_fence_after();
                    mma_tiles<D>(tmem_base + Cfg::T_S, q_s, sb + Cfg::OFF_K + (m % NK) * Cfg::TILE_BYTES, Cfg::IDESC_S);
                    mma_commit(s_full);
                    if (!w.wait(v_full((int)(m % NV)), (m / NV) & 1u, kDevErrMmaFull)) return false;
                    tcgen05_fence_after();
                    mma_tiles<D>(tmem_base + Cfg::T_DP + (m & 1u) * 128, o_s, sb + Cfg::OFF_V + (m % NV) * Cfg::TILE_BYTES, Cfg::IDESC_S);
                    mma_commit(dp_full((int)(m & 1u)));
                    mma_commit(v_empty((int)(m % NV)));
                    return true;
                };
                while (ok) {
                    const uint32_t box = n_box & 1u;
                    if (!w.wait(item_pub(box), (n_box >> 1) & 1u, kDevErrMmaFull)) break;
                    const Item it = read_item(box);
                    mbar_arrive(item_read(box));
                    ++n_box;
                    if (it.b < 0) break;
                    const int steps = it.t1 - it.t0;
                    if (steps <= 0) continue;
                    if (!w.wait(q_full, n_item & 1u, kDevErrMmaFull)) break;
                    ++n_item;
                    // the step before an item's first has been read too: its dS was waited for
                    if (!(ok = issue_scores(n, n == 0))) break;
                    for (int i = 0; i < steps; ++i, ++n) {
                        if (i + 1 < steps && !(ok = issue_scores(n + 1, false))) break;
                        if (!(ok = w.wait(ds_full((int)(n & 1u)), (n >> 1) & 1u, kDevErrMmaFull))) break;
                        tcgen05_fence_after();
                        mma_overlay(tmem_base + Cfg::T_DQ, tmem_base + Cfg::T_DP + (n & 1u) * 128,
                                    sb + Cfg::OFF_K + (n % NK) * Cfg::TILE_BYTES, Cfg::IDESC_ACC, i > 0);
                        mma_commit(k_empty((int)(n % NK)));
                    }
                    if (!ok) break;
                    mma_commit(q_empty);
                    mma_commit(done);
                }
                mma_commit(drain);
                w.drain(drain, 0);
            }
            __syncwarp();
        }
    } else {
        reg_inc<kBwdMathRegs>();
        // ------------------------------------------------------------ dS and the output (warps 4-11)
        const int half = (warp - 4) >> 2;                // key columns 64 half .. + 63
        const int quad = warp & 3;
        const int r = quad * 32 + lane;                  // query of the tile
        const uint32_t lane_base = tmem_base + ((uint32_t)(quad * 32) << 16);
        const uint32_t s_col = lane_base + Cfg::T_S + half * 64;
        uint32_t n_box = 0, n = 0, n_done = 0;
        bool ok = true;
        while (ok) {
            const uint32_t box = n_box & 1u;
            if (!__all_sync(0xffffffffu, w.wait(item_pub(box), (n_box >> 1) & 1u, kDevErrEpilogueFull))) break;
            const Item it = read_item(box);
            __syncwarp();
            if (lane == 0) mbar_arrive(item_read(box));
            ++n_box;
            if (it.b < 0) break;
            const int qi = it.q_base + r;                // below Sp
            const long long row = ((long long)it.b * mk.Hq + it.h) * p.Sp + qi;
            int lo = 0, hi = INT_MAX;                    // rows behind the last: no mask
            if (qi < mk.Sq) row_interval(mk, it.b, qi, lo, hi);
            const float shift = Elem<T>::bf16 ? 0.0f : ds_shift<T, Cfg::MODE>(__ldcg(p.row_norms + row), v_norm(p, it.b, it.h / mk.group, lane));
            const float off = __ldcg(p.offset + row) + shift, neg_delta = __ldcg(p.neg_delta + row);
            const float slope2 = kHasBias<Cfg::MODE> ? __ldg(p.score.slopes + it.h) * kLog2e : 0.0f;
            for (int t = it.t0; t < it.t1; ++t, ++n) {
                const int k0 = t * kTile + half * 64;
                const bool masked = __any_sync(0xffffffffu, k0 < lo || k0 + 64 > hi);
                if (!__all_sync(0xffffffffu, w.wait(s_full, n & 1u, kDevErrEpilogueFull))) {
                    ok = false;
                    break;
                }
                tcgen05_fence_after();
                uint32_t w0[32], w1[32], none[16];
                tmem_ld_32x32b_x32(s_col, w0);
                tmem_ld_32x32b_x32(s_col + 32, w1);
                tmem_ld_wait(w0);
                reg_tie(w1);
                tcgen05_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_read);
                if (masked && __builtin_expect(products_not_finite(w0, w1, nullptr, lane), 0)) {
                    if (clean_half_tile<T, DCH>(smem + Cfg::OFF_K + (n % NK) * Cfg::TILE_BYTES, half, lane)) cleaned[n_box & 3u] = n_box;
                    fence_proxy_async_smem();
                    if (kHasCap<Cfg::MODE>) {            // a hidden NaN would take its visible neighbour along
                        const uint32_t v0 = between(lo - k0, hi - k0), v1 = between(lo - k0 - 32, hi - k0 - 32);
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            if (!(v0 >> i & 1u)) w0[i] = 0u;
                            if (!(v1 >> i & 1u)) w1[i] = 0u;
                        }
                    }
                }
                const float base = (float)(qi + mk.offset - k0);
                auto offset = [&](int) { return make_float2(off, off); };
                weights_chunk<T, Cfg::MODE, false>(w0, p.score, slope2, base, offset, none);
                weights_chunk<T, Cfg::MODE, false>(w1, p.score, slope2, base - 32.0f, offset, none);
                const int buf = (int)(n & 1u);
                if (!__all_sync(0xffffffffu, w.wait(dp_full(buf), (n >> 1) & 1u, kDevErrEpilogueFull))) {
                    ok = false;
                    break;
                }
                tcgen05_fence_after();
                const uint32_t dp_col = lane_base + Cfg::T_DP + buf * 128 + half * 64;
                uint32_t dp0[32], dp1[32];
                tmem_ld_32x32b_x32(dp_col, dp0);
                tmem_ld_32x32b_x32(dp_col + 32, dp1);
                tmem_ld_wait(dp0);
                reg_tie(dp1);
                auto ds_chunk = [&](const uint32_t (&ww)[32], const uint32_t (&dp)[32], int c) {
                    uint32_t packed[16];
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        float d0 = __uint_as_float(dp[i]), d1 = __uint_as_float(dp[i + 1]);
                        fadd2(d0, d1, neg_delta, neg_delta);
                        fmul2(d0, d1, d0, d1, __uint_as_float(ww[i]), __uint_as_float(ww[i + 1]));
                        packed[i / 2] = Elem<T>::pack(d0, d1);
                    }
                    if (masked) {
                        const uint32_t vis = between(lo - k0 - c * 32, hi - k0 - c * 32);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!(vis >> i & 1u)) packed[i / 2] &= i & 1 ? 0x0000ffffu : 0xffff0000u;
                    }
                    tmem_st_32x32b_x16(dp_col + c * 16, packed);
                };
                ds_chunk(w0, dp0, 0);
                ds_chunk(w1, dp1, 1);
                tmem_st_wait();
                tcgen05_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(ds_full(buf));
            }
            if (!ok) break;
            const bool none = it.t0 >= it.t1;
            if (!none) {
                ok = __all_sync(0xffffffffu, w.wait(done, n_done & 1u, kDevErrEpilogueFull));
                ++n_done;
                tcgen05_fence_after();
                if (!ok) break;
            }
            // half 0 writes the rows; the next item's products overwrite the accumulator only after its
            // next dS
            const bool empty = none || lo >= hi;
            T* out = static_cast<T*>(p.dQ.data) + it.b * p.dQ.batch + it.h * p.dQ.head + (long long)qi * p.dQ.row;
            const float factor = kCapFactor<Cfg::MODE> * p.score.scale * exp2f(-kPShift<T> - shift);
            if (half == 0) {
                store_accumulator<T, D>(lane_base + Cfg::T_DQ, factor, empty, qi < mk.Sq, out);
                if (__builtin_expect(cleaned[n_box & 3u] == n_box, 0)) spread_dq<T, D>(p, it.b, it.h, it.q_base, it.t0, it.t1);
            }
            tcgen05_fence_before();
        }
    }

    grid_wait();                                         // whoever waits for dQ waits for dK and dV too
    tcgen05_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tcgen05_fence_after();
        tmem_dealloc(tmem_base, 512);
    }
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------
// The rows, then dK and dV, then dQ, then the sums of parts.  dK's and dV's CTAs start while the rows' last ones
// finish, and wait for them (let in while rows are still to come, they take SMs from them: 8192 tokens in 4
// documents 401 us, so 414).  dQ's CTAs need the rows alone (finished when dK's and dV's CTAs have come past
// their wait, which is when dQ's may start) and fill the SMs that run out of dK and dV items.
template <class T, int D, int MODE>
cudaError_t launch_bwd_mode(const MaskedBwdMaps& tm, const MaskedBwdParams& p, cudaStream_t stream) {
    using Dkv = DkvCfg<T, D, MODE>;
    using Dq = DqCfg<T, D, MODE>;
    static std::atomic<uint64_t> dkv_done{0}, dq_done{0};
    const int k_items = (p.mask.Skv + kTile - 1) / kTile * p.mask.B * p.mask.Hkv * p.splits;
    const int q_items = p.Sp / kTile * p.mask.B * p.mask.Hq;
    cudaError_t e;
    if ((e = allow_smem(gsr_masked_dkv_kernel<Dkv>, Dkv::SMEM_BYTES, dkv_done)) != cudaSuccess ||
        (e = allow_smem(gsr_masked_dq_kernel<Dq>, Dq::SMEM_BYTES, dq_done)) != cudaSuccess ||
        (e = launch_early(gsr_masked_dkv_kernel<Dkv>, (unsigned)k_items, kBwdThreads, Dkv::SMEM_BYTES, stream, tm.q, tm.k, tm.v,
                          tm.dO, p)) != cudaSuccess ||
        (e = launch_early(gsr_masked_dq_kernel<Dq>, (unsigned)q_items, kBwdThreads, Dq::SMEM_BYTES, stream, tm.q, tm.k, tm.v,
                          tm.dO, p)) != cudaSuccess)
        return e;
    if (p.splits > 1) {
        const long long rows = 2ll * p.mask.B * p.mask.Hkv * p.mask.Skv;
        return launch_early(gsr_masked_dkv_sum_kernel<T, D>, (unsigned)((rows + 8 * kSumRows - 1) / (8 * kSumRows)), 256, 0,
                            stream, p);
    }
    return cudaSuccess;
}

template <class T, int D>
cudaError_t launch_bwd_type(const MaskedBwdMaps& tm, const MaskedBwdParams& p, cudaStream_t stream) {
    const MaskArgs& mk = p.mask;
    const long long q_rows = (long long)mk.B * mk.Hq * mk.Sq, k_rows = (long long)mk.B * mk.Hkv * mk.Skv;
    if (q_rows == 0 || k_rows == 0) {                    // no pairs: every gradient is zero
        if (k_rows > 0) {
            const unsigned grid = (unsigned)((k_rows + 7) / 8);
            gsr_masked_zero_kernel<T, D><<<grid, 256, 0, stream>>>(p.dK, mk.Hkv, mk.Skv, k_rows);
            gsr_masked_zero_kernel<T, D><<<grid, 256, 0, stream>>>(p.dV, mk.Hkv, mk.Skv, k_rows);
        }
        if (q_rows > 0)
            gsr_masked_zero_kernel<T, D><<<(unsigned)((q_rows + 7) / 8), 256, 0, stream>>>(p.dQ, mk.Hq, mk.Sq, q_rows);
        return cudaGetLastError();
    }
    long long ctas = (long long)mk.B * mk.Hq * (p.Sp / kNormRows);
    if (!Elem<T>::bf16) ctas += (long long)mk.B * mk.Hkv * ((mk.Skv + kNormRows - 1) / kNormRows);
    gsr_masked_bwd_rows_kernel<T, D><<<(unsigned)ctas, 256, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    switch (score_mode(p.score)) {
        case kScorePlain: return launch_bwd_mode<T, D, kScorePlain>(tm, p, stream);
        case kScoreBias: return launch_bwd_mode<T, D, kScoreBias>(tm, p, stream);
        case kScoreCap: return launch_bwd_mode<T, D, kScoreCap>(tm, p, stream);
        default: return launch_bwd_mode<T, D, kScoreCapBias>(tm, p, stream);
    }
}

}  // namespace gsr
