// attention_masked_fwd.cu - attention forward with a document or prefix mask, capped scores, a
// distance bias and grouped heads:  O = softmax(score(Q K^T)) V.
#include "attention_common.cuh"

namespace gsr {
namespace {

// One query row by one warp.
template <class T, int D>
__device__ __forceinline__ void masked_row(const MaskedFwdParams& p, int b, int h, int i, int lane) {
    const int hk = h / p.mask.group;
    float q[D / 32], acc[D / 32], m, l;
    load_row<T, D>(static_cast<const T*>(p.Q.data) + b * p.Q.batch + h * p.Q.head + i * p.Q.row, lane, q);
    const T* kb = static_cast<const T*>(p.K.data) + b * p.K.batch + hk * p.K.head;
    const T* vb = static_cast<const T*>(p.V.data) + b * p.V.batch + hk * p.V.head;
    const float slope2 = p.score.slopes ? __ldg(p.score.slopes + h) * kLog2e : 0.0f;
    int lo, hi;
    row_interval(p.mask, b, i, lo, hi);
    const int pos = i + p.mask.offset;
    row_forward<T, D>(q, lo, hi, p.score, slope2, lane,
                      [&](int j, const T*& k, const T*& v, float& dist) {
                          k = kb + j * p.K.row;
                          v = vb + j * p.V.row;
                          dist = fabsf((float)(pos - j));
                          return true;
                      },
                      acc, m, l);
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) acc[e] *= inv;
    store_row<T, D>(static_cast<T*>(p.O.data) + b * p.O.batch + h * p.O.head + i * p.O.row, lane, acc);
    if (p.lse && lane == 0)
        p.lse[((long long)b * p.mask.Hq + h) * p.mask.Sq + i] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <class T, int D>
__global__ void __launch_bounds__(256) gsr_masked_rows_kernel(const MaskedFwdParams p) {
    const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= (long long)p.mask.B * p.mask.Hq * p.mask.Sq) return;
    const int i = (int)(row % p.mask.Sq);
    const int bh = (int)(row / p.mask.Sq);
    masked_row<T, D>(p, bh / p.mask.Hq, bh % p.mask.Hq, i, threadIdx.x & 31);
}

template <class T, int D>
cudaError_t launch(const MaskedFwdParams& p, cudaStream_t stream) {
    const long long rows = (long long)p.mask.B * p.mask.Hq * p.mask.Sq;
    gsr_masked_rows_kernel<T, D><<<(unsigned)((rows + 7) / 8), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_masked_fwd(const MaskedFwdParams& p, int D, bool bf16, cudaStream_t stream) {
    if (bf16) return D == 64 ? launch<__nv_bfloat16, 64>(p, stream) : launch<__nv_bfloat16, 128>(p, stream);
    return D == 64 ? launch<__half, 64>(p, stream) : launch<__half, 128>(p, stream);
}

}  // namespace gsr
