// attention_masked_bwd.cu - gradients of attention with a document or prefix mask, capped scores,
// a distance bias and grouped heads.
//
// With P_ij = exp(y_ij - lse_i) from the forward pass's log-sum-exp and delta_i = dO_i . O_i,
//     dV_j = sum_i P_ij dO_i
//     dS_ij = P_ij (dO_i . V_j - delta_i) c_ij          c = 1 - tanh^2 with a cap, else 1
//     dQ_i = scale sum_j dS_ij K_j        dK_j = scale sum_i dS_ij Q_i
// dK and dV of a key/value head sum over the query heads of its group.  dQ is summed by the CTA
// that owns the queries and dK, dV by the one that owns the keys, each recomputing P and dS, so no
// result depends on the order of atomics.
#include "attention_common.cuh"

namespace gsr {
namespace {

// ---------------------------------------------------------------------------
// Rows: lse in log2 units, delta, intervals, and the norms that bound dS
// ---------------------------------------------------------------------------
// One warp per query row (b, h, i), rows padded to Sp, then one per value row.  Bound by the read
// of dO and O.  Maxima are order-free, so the atomics are deterministic.
template <class T, int D>
__global__ void __launch_bounds__(256) gsr_masked_bwd_rows_kernel(const MaskedBwdParams p) {
    const int lane = threadIdx.x & 31;
    const MaskArgs& mk = p.mask;
    const long long q_rows = (long long)mk.B * mk.Hq * p.Sp;
    long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row < q_rows) {
        const int i = (int)(row % p.Sp), bh = (int)(row / p.Sp), b = bh / mk.Hq, h = bh % mk.Hq;
        float lse2 = INFINITY, delta = 0.0f;
        int lo = mk.Skv, hi = mk.Skv;
        if (i < mk.Sq) {
            row_interval(mk, b, i, lo, hi);
            if (lo < hi) {
                float x[D / 32], y[D / 32];
                load_row<T, D>(static_cast<const T*>(p.dO.data) + b * p.dO.batch + h * p.dO.head + i * p.dO.row, lane, x);
                load_row<T, D>(static_cast<const T*>(p.O.data) + b * p.O.batch + h * p.O.head + i * p.O.row, lane, y);
                delta = warp_dot(x, y);
                const float n = warp_dot(x, x);
                lse2 = __ldg(p.lse + ((long long)b * mk.Hq + h) * mk.Sq + i) * kLog2e;
                if (lse2 == -INFINITY) lse2 = INFINITY;
                if (lane == 0 && n < INFINITY) atomicMax(p.norms, __float_as_uint(n));
            }
        }
        if (lane == 0) {
            p.lse2[row] = lse2;
            p.delta[row] = delta;
            if (h == 0) {
                p.lo[(long long)b * p.Sp + i] = lo;
                p.hi[(long long)b * p.Sp + i] = hi;
            }
        }
        return;
    }
    row -= q_rows;
    if (row < (long long)mk.B * mk.Hkv * mk.Skv) {
        const int j = (int)(row % mk.Skv), bh = (int)(row / mk.Skv), b = bh / mk.Hkv, h = bh % mk.Hkv;
        float x[D / 32];
        load_row<T, D>(static_cast<const T*>(p.V.data) + b * p.V.batch + h * p.V.head + j * p.V.row, lane, x);
        const float n = warp_dot(x, x);
        if (lane == 0 && n < INFINITY) atomicMax(p.norms + 1, __float_as_uint(n));
    }
}

// P_ij and dS_ij of one pair, by one warp.
template <class T, int D>
__device__ __forceinline__ void pair_grad(const ScoreArgs& sc, float slope2, int dist, const float (&q)[D / 32],
                                          const float (&k)[D / 32], const float (&dO)[D / 32],
                                          const float (&v)[D / 32], float lse2, float delta, float& P, float& dS) {
    float grad;
    const float y = score_of(warp_dot(q, k), sc, grad) - slope2 * fabsf((float)dist);
    P = ex2_approx(y - lse2);
    dS = P * (warp_dot(dO, v) - delta) * grad;
}

// dQ of one query row, by one warp.
template <class T, int D>
__device__ __forceinline__ void row_dq(const MaskedBwdParams& p, int b, int h, int i, int lane) {
    const MaskArgs& mk = p.mask;
    const int hk = h / mk.group;
    float q[D / 32], dO[D / 32], k[D / 32], v[D / 32], acc[D / 32] = {};
    load_row<T, D>(static_cast<const T*>(p.Q.data) + b * p.Q.batch + h * p.Q.head + i * p.Q.row, lane, q);
    load_row<T, D>(static_cast<const T*>(p.dO.data) + b * p.dO.batch + h * p.dO.head + i * p.dO.row, lane, dO);
    const T* kb = static_cast<const T*>(p.K.data) + b * p.K.batch + hk * p.K.head;
    const T* vb = static_cast<const T*>(p.V.data) + b * p.V.batch + hk * p.V.head;
    const float slope2 = p.score.slopes ? __ldg(p.score.slopes + h) * kLog2e : 0.0f;
    const long long row = ((long long)b * mk.Hq + h) * p.Sp + i;
    const float lse2 = p.lse2[row], delta = p.delta[row];
    const int lo = p.lo[(long long)b * p.Sp + i], hi = p.hi[(long long)b * p.Sp + i];
    for (int j = lo; j < hi; ++j) {
        load_row<T, D>(kb + j * p.K.row, lane, k);
        load_row<T, D>(vb + j * p.V.row, lane, v);
        float P, dS;
        pair_grad<T, D>(p.score, slope2, i + mk.offset - j, q, k, dO, v, lse2, delta, P, dS);
#pragma unroll
        for (int e = 0; e < D / 32; ++e) acc[e] = fmaf(dS, k[e], acc[e]);
    }
#pragma unroll
    for (int e = 0; e < D / 32; ++e) acc[e] *= p.score.scale;
    store_row<T, D>(static_cast<T*>(p.dQ.data) + b * p.dQ.batch + h * p.dQ.head + i * p.dQ.row, lane, acc);
}

// dK and dV of one key row, by one warp: the queries that see key j are those from the first
// whose interval ends behind it to the first whose interval starts behind it.
template <class T, int D>
__device__ __forceinline__ void row_dkv(const MaskedBwdParams& p, int b, int hk, int j, int lane) {
    const MaskArgs& mk = p.mask;
    float q[D / 32], dO[D / 32], k[D / 32], v[D / 32], dk[D / 32] = {}, dv[D / 32] = {};
    load_row<T, D>(static_cast<const T*>(p.K.data) + b * p.K.batch + hk * p.K.head + j * p.K.row, lane, k);
    load_row<T, D>(static_cast<const T*>(p.V.data) + b * p.V.batch + hk * p.V.head + j * p.V.row, lane, v);
    const int* los = p.lo + (long long)b * p.Sp;
    const int* his = p.hi + (long long)b * p.Sp;
    int begin = 0, end = mk.Sq;
    for (int right = mk.Sq; begin < right;) {
        const int mid = (begin + right) >> 1;
        if (his[mid] <= j) begin = mid + 1;
        else right = mid;
    }
    for (int left = begin; left < end;) {
        const int mid = (left + end) >> 1;
        if (los[mid] <= j) left = mid + 1;
        else end = mid;
    }
    for (int h = hk * mk.group; h < (hk + 1) * mk.group; ++h) {
        const T* qb = static_cast<const T*>(p.Q.data) + b * p.Q.batch + h * p.Q.head;
        const T* ob = static_cast<const T*>(p.dO.data) + b * p.dO.batch + h * p.dO.head;
        const float slope2 = p.score.slopes ? __ldg(p.score.slopes + h) * kLog2e : 0.0f;
        const long long row = ((long long)b * mk.Hq + h) * p.Sp;
        for (int i = begin; i < end; ++i) {
            if (j < los[i] || j >= his[i]) continue;
            load_row<T, D>(qb + i * p.Q.row, lane, q);
            load_row<T, D>(ob + i * p.dO.row, lane, dO);
            float P, dS;
            pair_grad<T, D>(p.score, slope2, i + mk.offset - j, q, k, dO, v, p.lse2[row + i], p.delta[row + i], P, dS);
#pragma unroll
            for (int e = 0; e < D / 32; ++e) {
                dv[e] = fmaf(P, dO[e], dv[e]);
                dk[e] = fmaf(dS, q[e], dk[e]);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < D / 32; ++e) dk[e] *= p.score.scale;
    store_row<T, D>(static_cast<T*>(p.dK.data) + b * p.dK.batch + hk * p.dK.head + j * p.dK.row, lane, dk);
    store_row<T, D>(static_cast<T*>(p.dV.data) + b * p.dV.batch + hk * p.dV.head + j * p.dV.row, lane, dv);
}

template <class T, int D>
__global__ void __launch_bounds__(256) gsr_masked_dq_kernel(const MaskedBwdParams p) {
    const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= (long long)p.mask.B * p.mask.Hq * p.mask.Sq) return;
    const int bh = (int)(row / p.mask.Sq);
    row_dq<T, D>(p, bh / p.mask.Hq, bh % p.mask.Hq, (int)(row % p.mask.Sq), threadIdx.x & 31);
}

template <class T, int D>
__global__ void __launch_bounds__(256) gsr_masked_dkv_kernel(const MaskedBwdParams p) {
    const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= (long long)p.mask.B * p.mask.Hkv * p.mask.Skv) return;
    const int bh = (int)(row / p.mask.Skv);
    row_dkv<T, D>(p, bh / p.mask.Hkv, bh % p.mask.Hkv, (int)(row % p.mask.Skv), threadIdx.x & 31);
}

template <class T, int D>
cudaError_t launch(const MaskedBwdParams& p, cudaStream_t stream) {
    const MaskArgs& mk = p.mask;
    const long long q_rows = (long long)mk.B * mk.Hq * mk.Sq, k_rows = (long long)mk.B * mk.Hkv * mk.Skv;
    const long long rows = (long long)mk.B * mk.Hq * p.Sp + k_rows;
    cudaError_t e = cudaMemsetAsync(p.norms, 0, 2 * sizeof(unsigned), stream);
    if (e != cudaSuccess) return e;
    gsr_masked_bwd_rows_kernel<T, D><<<(unsigned)((rows + 7) / 8), 256, 0, stream>>>(p);
    if (k_rows > 0) gsr_masked_dkv_kernel<T, D><<<(unsigned)((k_rows + 7) / 8), 256, 0, stream>>>(p);
    if (q_rows > 0) gsr_masked_dq_kernel<T, D><<<(unsigned)((q_rows + 7) / 8), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_masked_bwd(const MaskedBwdParams& p, int D, bool bf16, cudaStream_t stream) {
    if (bf16) return D == 64 ? launch<__nv_bfloat16, 64>(p, stream) : launch<__nv_bfloat16, 128>(p, stream);
    return D == 64 ? launch<__half, 64>(p, stream) : launch<__half, 128>(p, stream);
}

}  // namespace gsr
