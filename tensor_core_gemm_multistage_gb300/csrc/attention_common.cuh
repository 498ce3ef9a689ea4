// attention_common.cuh - what the masked, backward and tree attention kernels share: element
// types, the interval of keys a query sees, the score function, and attention of single rows.
#pragma once

#include <atomic>

#include <cuda_bf16.h>

#include "device_common.cuh"
#include "llm.h"

namespace gsr {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ---------------------------------------------------------------------------
// fp16 and bf16
// ---------------------------------------------------------------------------
template <class T>
struct Elem;
template <>
struct Elem<__half> {
    static constexpr bool bf16 = false;
    static __device__ __forceinline__ float2 unpack(uint32_t v) {
        return __half22float2(*reinterpret_cast<const __half2*>(&v));
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static constexpr uint32_t exponent = 0x7c00u;        // all of its bits set: infinite or NaN
    // acc + 0 v: NaN from the first v on that is not finite
    static __device__ __forceinline__ uint32_t fma_zero(uint32_t v, uint32_t acc) {
        const __half2 h = __hfma2(*reinterpret_cast<const __half2*>(&v), __half2half2(__ushort_as_half(0)),
                                  *reinterpret_cast<const __half2*>(&acc));
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};
template <>
struct Elem<__nv_bfloat16> {
    static constexpr bool bf16 = true;
    static __device__ __forceinline__ float2 unpack(uint32_t v) {
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static constexpr uint32_t exponent = 0x7f80u;
    static __device__ __forceinline__ uint32_t fma_zero(uint32_t v, uint32_t acc) {
        const __nv_bfloat162 h = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v), __bfloat162bfloat162(__ushort_as_bfloat16(0)),
                                         *reinterpret_cast<const __nv_bfloat162*>(&acc));
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};

// ---------------------------------------------------------------------------
// The keys a query sees: one interval [lo, hi)
// ---------------------------------------------------------------------------
// A document mask keeps [start, end) of the query's own document; a causal mask ends the interval
// behind the query's position p, a prefix behind the prefix if that is later.  With boundaries in
// ascending order lo and hi never fall from one query to the next, so the keys of a block of
// queries are [lo of its first, hi of its last).  A query outside every document gets an empty
// interval at the nearest boundary, which keeps that order.
__device__ __forceinline__ void row_interval(const MaskArgs& m, int b, int i, int& lo, int& hi) {
    int s = 0, e = m.Skv, d = 0;
    if (m.num_docs > 0) {
        const int* bounds = m.doc_bounds + (long long)b * (m.num_docs + 1);
        int left = 0, right = m.num_docs + 1;          // first boundary above i
        while (left < right) {
            const int mid = (left + right) >> 1;
            if (__ldg(bounds + mid) <= i) left = mid + 1;
            else right = mid;
        }
        d = left - 1;
        if (d < 0 || d >= m.num_docs) {
            lo = hi = min(max(__ldg(bounds + (d < 0 ? 0 : m.num_docs)), 0), m.Skv);
            return;
        }
        s = max(__ldg(bounds + d), 0);
        e = min(__ldg(bounds + d + 1), m.Skv);
    }
    lo = s;
    hi = e;
    if (m.causal) {
        int limit = i + m.offset + 1;
        if (m.prefix_lens) {
            const long long n = m.num_docs > 0 ? m.num_docs : 1;
            limit = max(limit, s + min(max(__ldg(m.prefix_lens + b * n + d), 0), m.Skv - s));
        }
        hi = min(e, limit);
    }
    hi = max(hi, lo);
}

// The other way round: the queries that see key j are the interval [first, end).
__device__ __forceinline__ void key_interval(const MaskArgs& m, int b, int j, int& first, int& end) {
    int s = 0, d = 0;
    first = 0;
    end = m.Sq;
    if (m.num_docs > 0) {                              // offset 0: documents need Sq == Skv
        const int* bounds = m.doc_bounds + (long long)b * (m.num_docs + 1);
        int left = 0, right = m.num_docs + 1;          // first boundary above j
        while (left < right) {
            const int mid = (left + right) >> 1;
            if (__ldg(bounds + mid) <= j) left = mid + 1;
            else right = mid;
        }
        d = left - 1;
        if (d < 0 || d >= m.num_docs) {
            first = end = min(max(__ldg(bounds + (d < 0 ? 0 : m.num_docs)), 0), m.Sq);
            return;
        }
        s = first = max(__ldg(bounds + d), 0);
        end = min(__ldg(bounds + d + 1), m.Sq);
    }
    if (m.causal) {
        bool all = false;
        if (m.prefix_lens) {
            const long long n = m.num_docs > 0 ? m.num_docs : 1;
            all = j < s + min(max(__ldg(m.prefix_lens + b * n + d), 0), m.Skv - s);
        }
        if (!all) first = max(first, min(j - m.offset, m.Sq));
    }
    end = max(end, first);
}

// Bits [from, to) of 32.
__device__ __forceinline__ uint32_t between(int from, int to) {
    auto below = [](int n) { return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u); };
    return below(to) & ~below(from);
}

// ---------------------------------------------------------------------------
// Scores
// ---------------------------------------------------------------------------
// rcp.approx: within 1 ulp; +inf gives 0.
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// tanh(x) = 1 - 2 / (1 + e^(2x)): with r = 1 / (1 + 2^(cap_in s)) the capped score is
// cap_out (1 - 2 r), and tanh's derivative 4 r (1 - r) has no cancellation.  The absolute error
// of a score is a few units of cap 2^-24, which is what the softmax sees.
//
// Capped scores of a row are taken through z = (8/3) scale q.k / cap, so that bit 30 of a z, set where
// its magnitude is 2 or more (or it is infinite or NaN), says that the tanh's argument is beyond 3/4.
//
// tanh(3/8 z) for |z| < 2, two values in place: z times a polynomial in z^2, whose six coefficients
// minimise the largest relative error over the range (3e-8; a weighted least-squares fit with the
// weights moved to where the error is).  Off by 1e-7 at most in fp32.  Seven FMA slots a score, where
// 1 / (1 + e^(2x)) takes an exponential and a reciprocal, three slots of the exponential's size on the
// special-function unit (32 and 16 a clock and SM, measured), which two softmax groups share with the
// probabilities' exponentials (4 x 32 x 4096 x 128 capped, forward: 1116 us, 1345 without it).
__device__ __forceinline__ void tanh_small2(float& z0, float& z1) {
    float u0, u1, p0, p1;
    fmul2(u0, u1, z0, z1, z0, z1);
    ffma2(p0, p1, u0, u1, -9.72615837e-08f, -9.72615837e-08f, 2.87182866e-06f, 2.87182866e-06f);
    ffma2(p0, p1, p0, p1, u0, u1, -5.5629851e-05f, -5.5629851e-05f);
    ffma2(p0, p1, p0, p1, u0, u1, 0.00098818168f, 0.00098818168f);
    ffma2(p0, p1, p0, p1, u0, u1, -0.0175779276f, -0.0175779276f);
    ffma2(p0, p1, p0, p1, u0, u1, 0.375f, 0.375f);
    fmul2(z0, z1, z0, z1, p0, p1);
}
// The same for any z: 1 - 2 r.
__device__ __forceinline__ void tanh_any2(float& z0, float& z1) {
    constexpr float kExponent = 2.0f * 0.375f * kLog2e;
    fmul2(z0, z1, z0, z1, kExponent, kExponent);
    z0 = ex2_approx(z0);
    z1 = ex2_approx(z1);
    fadd2(z0, z1, 1.0f, 1.0f);
    z0 = rcp_approx(z0);
    z1 = rcp_approx(z1);
    ffma2(z0, z1, z0, z1, -2.0f, -2.0f, 1.0f, 1.0f);
}
// 32 products -> z in place; returns the bits set in any of them.
__device__ __forceinline__ uint32_t cap_scale(uint32_t (&rr)[32], float cap_z) {
    uint32_t bits = 0u;
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
        float y0, y1;
        fmul2(y0, y1, __uint_as_float(rr[i]), __uint_as_float(rr[i + 1]), cap_z, cap_z);
        rr[i] = __float_as_uint(y0);
        rr[i + 1] = __float_as_uint(y1);
        bits |= rr[i] | rr[i + 1];
    }
    return bits;
}

// r of two products, in place, with one reciprocal, 1 / a = b / (a b).  2^60 keeps a b finite and is
// tanh = 1 to the last bit.  A NaN stays one and takes its partner along: hidden products that are not
// finite are set to 0 first.  For the gradients' kernels, whose special-function unit has room (4 x 32 x 4096 x 128
// capped: 3287 us, 3488 with two reciprocals; the polynomial, in two copies of the code, was slower
// than either).
__device__ __forceinline__ float min_nan(float a, float b) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ void cap_r_pair(float& s0, float& s1, float cap_in) {
    float a, b;
    fmul2(a, b, s0, s1, cap_in, cap_in);
    a = ex2_approx(min_nan(a, 60.0f));
    b = ex2_approx(min_nan(b, 60.0f));
    fadd2(a, b, 1.0f, 1.0f);
    const float r = rcp_approx(a * b);
    fmul2(s0, s1, r, r, b, a);
}
enum ScoreMode : int { kScorePlain = 0, kScoreBias = 1, kScoreCap = 2, kScoreCapBias = 3 };
template <int MODE>
constexpr bool kHasCap = MODE == kScoreCap || MODE == kScoreCapBias;
template <int MODE>
constexpr bool kHasBias = MODE == kScoreBias || MODE == kScoreCapBias;
inline ScoreMode score_mode(const ScoreArgs& sc) {
    return sc.cap_in != 0.0f ? (sc.slopes ? kScoreCapBias : kScoreCap) : (sc.slopes ? kScoreBias : kScorePlain);
}

// A row's scores while its softmax runs: registers hold v with score = mul v in log2 units, so
// that the scaling is part of the exponent's multiply-add.  Plain scores keep the raw products;
// capped ones without a bias keep the tanh; anything with a bias holds the score itself.  A score's
// order is v's where mul >= 0 and the reverse elsewhere.
struct ScoreForm {
    float mul;
    bool ascending;
    __device__ __forceinline__ uint32_t hidden() const { return ascending ? 0xff800000u : 0x7f800000u; }   // score -inf
};
template <int MODE>
__device__ __forceinline__ ScoreForm score_form(const ScoreArgs& sc) {
    if (MODE == kScorePlain) return {sc.sl2, sc.sl2 >= 0.0f};
    if (MODE == kScoreCap) return {sc.cap_out, true};
    return {1.0f, true};
}

// 32 raw products of one row and consecutive keys -> v, in place.  `base` is the first key's
// distance from the row's position (later keys are closer by 1 each).  With a cap the registers hold
// z; SMALL: every z of the row is below 2.
template <int MODE, bool SMALL>
__device__ __forceinline__ void score_chunk(uint32_t (&rr)[32], const ScoreArgs& sc, float slope2, float base) {
    if (MODE == kScorePlain) return;
    if (MODE == kScoreBias && base >= 31.0f) {           // no key behind the row: the bias is linear
        const float at0 = -slope2 * base;
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            float w0, w1, y0 = __uint_as_float(rr[i]), y1 = __uint_as_float(rr[i + 1]);
            ffma2(w0, w1, slope2, slope2, (float)i, (float)(i + 1), at0, at0);
            ffma2(y0, y1, y0, y1, sc.sl2, sc.sl2, w0, w1);
            rr[i] = __float_as_uint(y0);
            rr[i + 1] = __float_as_uint(y1);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
        float y0 = __uint_as_float(rr[i]), y1 = __uint_as_float(rr[i + 1]);
        if (kHasCap<MODE> && SMALL) {
            tanh_small2(y0, y1);
        } else if (kHasCap<MODE>) {
            tanh_any2(y0, y1);
        } else {
            fmul2(y0, y1, y0, y1, sc.sl2, sc.sl2);
        }
        if (kHasBias<MODE>) {
            if (kHasCap<MODE>) fmul2(y0, y1, y0, y1, sc.cap_out, sc.cap_out);
            y0 = fmaf(-slope2, fabsf(base - (float)i), y0);
            y1 = fmaf(-slope2, fabsf(base - (float)(i + 1)), y1);
        }
        rr[i] = __float_as_uint(y0);
        rr[i + 1] = __float_as_uint(y1);
    }
}

// A launch whose CTAs may start before the launch ahead of it on the stream has finished (they wait
// for it themselves, grid_wait).
template <class... Params, class... Args>
cudaError_t launch_early(void (*kernel)(Params...), unsigned grid, unsigned block, int smem, cudaStream_t stream,
                         const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// A row's 128 products.  With POLY the warp takes tanh's polynomial where all its rows may.
template <int MODE, bool POLY>
__device__ __forceinline__ void score_row(uint32_t (&a)[32], uint32_t (&b)[32], uint32_t (&c)[32], uint32_t (&d)[32],
                                          const ScoreArgs& sc, float slope2, float base) {
    if (MODE == kScorePlain) return;
    if (kHasCap<MODE>) {
        const uint32_t bits = cap_scale(a, sc.cap_z) | cap_scale(b, sc.cap_z) | cap_scale(c, sc.cap_z) | cap_scale(d, sc.cap_z);
        if (POLY && __all_sync(0xffffffffu, !(bits & 0x40000000u))) {
            score_chunk<MODE, true>(a, sc, slope2, base);
            score_chunk<MODE, true>(b, sc, slope2, base - 32.0f);
            score_chunk<MODE, true>(c, sc, slope2, base - 64.0f);
            score_chunk<MODE, true>(d, sc, slope2, base - 96.0f);
            return;
        }
    }
    score_chunk<MODE, false>(a, sc, slope2, base);
    score_chunk<MODE, false>(b, sc, slope2, base - 32.0f);
    score_chunk<MODE, false>(c, sc, slope2, base - 64.0f);
    score_chunk<MODE, false>(d, sc, slope2, base - 96.0f);
}

// Largest and smallest of a row's 128 values, in four chains of three-input instructions.
__device__ __forceinline__ float row_max(const uint32_t (&a)[32], const uint32_t (&b)[32], const uint32_t (&c)[32],
                                         const uint32_t (&d)[32]) {
    float e0 = -INFINITY, e1 = e0, e2 = e0, e3 = e0;
    auto fold = [&](const uint32_t (&rr)[32]) {
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
            e0 = max3f(e0, __uint_as_float(rr[i]), __uint_as_float(rr[i + 1]));
            e1 = max3f(e1, __uint_as_float(rr[i + 2]), __uint_as_float(rr[i + 3]));
            e2 = max3f(e2, __uint_as_float(rr[i + 4]), __uint_as_float(rr[i + 5]));
            e3 = max3f(e3, __uint_as_float(rr[i + 6]), __uint_as_float(rr[i + 7]));
        }
    };
    fold(a);
    fold(b);
    fold(c);
    fold(d);
    return max3f(fmaxf(e0, e1), e2, e3);
}
__device__ __forceinline__ float row_min(const uint32_t (&a)[32], const uint32_t (&b)[32], const uint32_t (&c)[32],
                                         const uint32_t (&d)[32]) {
    float e0 = INFINITY, e1 = e0, e2 = e0, e3 = e0;
    auto fold = [&](const uint32_t (&rr)[32]) {
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
            e0 = min3f(e0, __uint_as_float(rr[i]), __uint_as_float(rr[i + 1]));
            e1 = min3f(e1, __uint_as_float(rr[i + 2]), __uint_as_float(rr[i + 3]));
            e2 = min3f(e2, __uint_as_float(rr[i + 4]), __uint_as_float(rr[i + 5]));
            e3 = min3f(e3, __uint_as_float(rr[i + 6]), __uint_as_float(rr[i + 7]));
        }
    };
    fold(a);
    fold(b);
    fold(c);
    fold(d);
    return min3f(fminf(e0, e1), e2, e3);
}

// Once per device: lets `kernel` use `bytes` of dynamic shared memory.
template <class K>
cudaError_t allow_smem(K* kernel, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_acq_rel);
    return e;
}

// ---------------------------------------------------------------------------
// Infinities and NaN behind a mask
// ---------------------------------------------------------------------------
// A masked pair has weight 0 in the matrix products, and 0 times an infinity or NaN would put a NaN into
// a result that does not see it.  In a tile that not every row of the product sees whole (an edge; elsewhere
// nothing is hidden), the elements of the weighted operand that are not finite are set to zero in
// shared memory before the product.  What they mean to the rows that do see them is added after the
// rows have been written: there a column with such an element is infinite or NaN, whatever its weight.
// Both steps cost by the tile and not by the pair, so a call with infinities takes about as long as one
// without.

// Whether 16-byte pieces in shared memory, a multiple of 256, hold something not finite.  By one warp.
template <class T>
__device__ __forceinline__ bool pieces_not_finite(const uint8_t* at, int pieces, int lane) {
    const uint4* p = reinterpret_cast<const uint4*>(at) + lane;
    uint32_t acc[4] = {0u, 0u, 0u, 0u};
    for (int i = 0; i < pieces; i += 256) {
        uint4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = p[i + 32 * k];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            acc[0] = Elem<T>::fma_zero(v[k].x, acc[0]);
            acc[1] = Elem<T>::fma_zero(v[k].y, acc[1]);
            acc[2] = Elem<T>::fma_zero(v[k].z, acc[2]);
            acc[3] = Elem<T>::fma_zero(v[k].w, acc[3]);
        }
    }
    return __any_sync(0xffffffffu, ((acc[0] | acc[1] | acc[2] | acc[3]) & (Elem<T>::exponent * 0x10001u)) != 0u);
}

// Sets what is not finite there to zero; true if there was something.  By one warp; the caller fences before the
// product.
template <class T>
__device__ __forceinline__ bool zero_not_finite(uint8_t* at, int pieces, int lane) {
    constexpr uint32_t E = Elem<T>::exponent;
    bool any = false;
#pragma unroll 1
    for (int i = lane; i < pieces; i += 32) {
        uint4 v = reinterpret_cast<uint4*>(at)[i];
        uint32_t* w = &v.x;
        bool found = false;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if ((w[k] & E) == E) {
                w[k] &= 0xffff0000u;
                found = true;
            }
            if ((w[k] >> 16 & E) == E) {
                w[k] &= 0x0000ffffu;
                found = true;
            }
        }
        if (found) reinterpret_cast<uint4*>(at)[i] = v;
        any |= found;
    }
    return __any_sync(0xffffffffu, any);
}

// One value more in a sum that is held rounded to T, or in fp32.
template <class T>
__device__ __forceinline__ void add_to(uint16_t* to, float x) {
    *to = (uint16_t)Elem<T>::pack(Elem<T>::unpack(*to).x + x, 0.0f);
}
template <class T>
__device__ __forceinline__ void add_to(float* to, float x) {
    *to += x;
}

// This lane's result row: which columns rows that it sees make +inf and -inf, both for NaN.
template <int D>
struct Marks {
    uint32_t plus[D / 32], minus[D / 32];
    __device__ __forceinline__ Marks() {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) plus[c] = minus[c] = 0u;
    }
    // A row of the weighted operand, one for the whole warp; `sees`: this lane's result row sees it.
    // NAN_ONLY: whatever is not finite there makes the column NaN (the weights are not finite either, or 0).
    template <class T, bool NAN_ONLY, int ROWS>
    __device__ __forceinline__ void take(const uint16_t (&x)[ROWS][D / 32], const bool (&sees)[ROWS]) {
        constexpr uint32_t E = Elem<T>::exponent;
#pragma unroll
        for (int k = 0; k < ROWS; ++k)
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                const uint32_t v = x[k][c];
                const bool special = (v & E) == E, nan = special && (NAN_ONLY || (v & 0x7fffu) != E);
                const uint32_t up = __ballot_sync(0xffffffffu, special && (nan || !(v & 0x8000u)));
                const uint32_t down = __ballot_sync(0xffffffffu, special && (nan || (v & 0x8000u)));
                if (sees[k]) {
                    plus[c] |= up;
                    minus[c] |= down;
                }
            }
    }
    // Into column blocks [c0, c1) of the row, which this lane has written; Out is uint16_t (a T) or float.
    template <class T, class Out>
    __device__ __forceinline__ void apply(Out* row, int c0 = 0, int c1 = D / 32) const {
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
            for (uint32_t bits = c >= c0 && c < c1 ? plus[c] | minus[c] : 0u; bits; bits &= bits - 1) {
                const int e = __ffs(bits) - 1;
                const float x = (plus[c] >> e & 1u) ? ((minus[c] >> e & 1u) ? NAN : INFINITY) : -INFINITY;
                add_to<T>(row + c * 32 + e, x);
            }
    }
};

// Whether one of rows [r0, r1), `pitch` elements apart, holds something not finite.  By one warp.
template <class T, int D>
__device__ __noinline__ bool rows_not_finite(const T* rows, long long pitch, int r0, int r1, int lane) {
    constexpr int PIECES = D / 8, ROWS = 32 / PIECES;    // 16-byte pieces of a row, rows at once
    uint32_t acc = 0u;
    rows += lane % PIECES * 8;
    for (int r = r0 + lane / PIECES; r < r1; r += 16 * ROWS) {
        uint4 x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = __ldg(reinterpret_cast<const uint4*>(rows + min(r + i * ROWS, r1 - 1) * pitch));
#pragma unroll
        for (int i = 0; i < 16; ++i)
            acc = Elem<T>::fma_zero(x[i].x, Elem<T>::fma_zero(x[i].y, Elem<T>::fma_zero(x[i].z, Elem<T>::fma_zero(x[i].w, acc))));
    }
    return __any_sync(0xffffffffu, (acc & (Elem<T>::exponent * 0x10001u)) != 0u);
}

// Rows [r0, r1) of the weighted operand (`pitch` elements apart), and this lane's result row, which sees those
// in [lo, hi) (`write`: it exists).  The whole warp calls it.
template <class T, int D, bool NAN_ONLY, class Out>
__device__ __noinline__ void spread_not_finite(const T* rows, long long pitch, int r0, int r1, int lo, int hi, Out* row, bool write,
                                               int lane) {
    if (!rows_not_finite<T, D>(rows, pitch, r0, r1, lane)) return;
    Marks<D> marks;
    for (int r = r0; r < r1; r += 4) {
        uint16_t x[4][D / 32];
        bool sees[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int at = min(r + k, r1 - 1);
            sees[k] = at >= lo && at < hi;
#pragma unroll
            for (int c = 0; c < D / 32; ++c)
                x[k][c] = __ldg(reinterpret_cast<const unsigned short*>(rows) + at * pitch + c * 32 + lane);
        }
        marks.template take<T, NAN_ONLY, 4>(x, sees);
    }
    if (write) marks.template apply<T>(row);
}

// ---------------------------------------------------------------------------
// Rows by one warp
// ---------------------------------------------------------------------------
// Lane t holds elements [t D/32, (t + 1) D/32) of a row.
template <class T, int D>
__device__ __forceinline__ void store_row(T* row, int lane, const float (&x)[D / 32]) {
    if constexpr (D == 128)
        reinterpret_cast<uint2*>(row)[lane] = make_uint2(Elem<T>::pack(x[0], x[1]), Elem<T>::pack(x[2], x[3]));
    else
        reinterpret_cast<uint32_t*>(row)[lane] = Elem<T>::pack(x[0], x[1]);
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

}  // namespace gsr
