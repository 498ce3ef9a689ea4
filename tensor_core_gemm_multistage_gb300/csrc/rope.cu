// rope.cu - norms of queries and keys for each head with the position rotation in the same pass, its
// gradient, and the writes of keys and values to a paged cache of 16 or 4 bits with both on the way.
//
// A row x of D values becomes rot(n w), n = x / sqrt(mean(x^2) + eps): pair (a, b) of the first R columns
// turns to (a c - b s, b c + a s).  Every row is read and written once and carries a few operations a byte,
// so the time is that of the bytes (4 D a row forwards, 6 D backwards), or of the launch.
//
// A row is held by D / 16 lanes in two 16-byte pieces each, chosen so that a lane has both halves of its
// pairs: nothing but the sums crosses lanes.  A warp takes one token's heads, so that the token's angles are
// loaded once for all of them (read for each row, they would be twice the row's bytes).
#include "rows16.cuh"
#include "serving.h"

namespace gsr {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

// What a lane holds of a row, and which angles go with it: 16-byte pieces c0 and c1; angles 8 first to 8 first + 7.
struct LanePart {
    int c0, c1;
    bool turns;
};
__device__ __forceinline__ LanePart lane_part(int l, int R, bool interleaved) {
    const int rc = R >> 4;                       // lanes with pairs
    if (interleaved || l >= rc) return {2 * l, 2 * l + 1, l < rc};
    return {l, l + rc, true};                    // column i turns with i + R / 2
}

// Each product and sum rounded by itself, so that codes of 4 bits do not hang on a contraction.
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
    const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    a = x;
}
// v[0..7] is piece c0, v[8..15] piece c1; `cosines` the lane's eight of its token, its sines R / 2 behind.  They are loaded for
// each row, from L1 after the first: held in registers they cost a third of the warps.
__device__ __forceinline__ void rotate(float (&v)[16], const float* cosines, int R, bool interleaved, float sign) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const float4 c4 = __ldg(reinterpret_cast<const float4*>(cosines) + half);
        const float4 s4 = __ldg(reinterpret_cast<const float4*>(cosines + R / 2) + half);
        const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = 4 * half + i;
            if (interleaved) turn(v[2 * k], v[2 * k + 1], c[i], sign * s[i]);
            else turn(v[k], v[8 + k], c[i], sign * s[i]);
        }
    }
}
template <int LANES>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
template <class T>
__device__ __forceinline__ void load_part(const T* row, const LanePart& at, uint4& lo, uint4& hi) {
    lo = reinterpret_cast<const uint4*>(row)[at.c0];     // not the read-only path: a call may work in place
    hi = reinterpret_cast<const uint4*>(row)[at.c1];
}
template <class T>
__device__ __forceinline__ void load_weight(const T* w, const LanePart& at, float (&to)[16]) {
    unpack8<T>(__ldg(reinterpret_cast<const uint4*>(w) + at.c0), to);
    unpack8<T>(__ldg(reinterpret_cast<const uint4*>(w) + at.c1), to + 8);
}
template <class T>
__device__ __forceinline__ void store_part(T* row, const LanePart& at, const float (&v)[16]) {
    reinterpret_cast<uint4*>(row)[at.c0] = pack8<T>(v);
    reinterpret_cast<uint4*>(row)[at.c1] = pack8<T>(v + 8);
}

// ---------------------------------------------------------------------------
// Forward, and the cache writes
// ---------------------------------------------------------------------------
enum Sink : int { kSinkRows, kSinkCache16, kSinkCache4 };

// Units of work: a token's heads in blocks of `per`, first those of Q, then K's, then (cache writes) V's.
struct RopePlan {
    Divider by_unit, by_seq, by_page;
    int per, q_blocks, k_blocks, units;
};

// A row of 4 bits: per 64 values minimum m and scale s = (maximum - m) / 15, both rounded to T, and codes
// rint((x - m) / s) cut to 0..15.  A group that holds infinities or NaN, or spans more than a float, is NaN as a whole.
template <class T, int D>
__device__ __forceinline__ void store_row4(const Cache4& cache, long long page, int row, int head, const LanePart& at, int l,
                                           bool live, const float (&v)[16]) {
    constexpr int LANES = D / 16;
    uint32_t words[2] = {0u, 0u}, pair[D / 64];
    float inv_m[D / 64], scale[D / 64];
#pragma unroll
    for (int g = 0; g < D / 64; ++g) {
        float lo = INFINITY, hi = -INFINITY, bad = 0.0f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (D > 64 && ((k ? at.c1 : at.c0) >> 3) != g) continue;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                lo = fminf(lo, v[8 * k + i]);
                hi = fmaxf(hi, v[8 * k + i]);
                bad = fmaf(v[8 * k + i], 0.0f, bad);        // NaN from an infinity or NaN
            }
        }
#pragma unroll
        for (int o = LANES / 2; o; o >>= 1) {
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
            bad += __shfl_xor_sync(0xffffffffu, bad, o);
        }
        const float span = (hi - lo) + bad;
        const float s = span <= 3.402823466e38f ? __fmul_rn(hi - lo, 1.0f / 15.0f) : NAN;
        pair[g] = Pair<T>::pack(s, s == s ? lo : NAN);
        const float2 held = Pair<T>::unpack(pair[g]);
        scale[g] = held.x;
        inv_m[g] = held.y;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int g = D > 64 ? (k ? at.c1 : at.c0) >> 3 : 0;
        const float s = D > 64 ? (g ? scale[D / 64 - 1] : scale[0]) : scale[0], m = D > 64 ? (g ? inv_m[D / 64 - 1] : inv_m[0]) : inv_m[0];
        if (s > 0.0f) {
            // the product with 1 / s is off by at most 2^-18 where the code is not cut: divided only next to a border
            const float inv = __frcp_rn(s);
            bool border = inv > 1.7e38f;
            uint32_t w = 0u;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = (v[8 * k + i] - m) * inv, c = rintf(x);
                border |= fabsf(x - c) > 0.4999f;
                w |= (uint32_t)fminf(fmaxf(c, 0.0f), 15.0f) << (4 * i);
            }
            if (border) {
                w = 0u;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    w |= (uint32_t)fminf(fmaxf(rintf(__fdiv_rn(v[8 * k + i] - m, s)), 0.0f), 15.0f) << (4 * i);
            }
            words[k] = w;
        }
    }
    if (!live) return;
    char* codes = cache.codes.data + page * cache.codes.page + (long long)row * cache.codes.row + head * cache.codes.head;
    reinterpret_cast<uint32_t*>(codes)[at.c0] = words[0];
    reinterpret_cast<uint32_t*>(codes)[at.c1] = words[1];
    if (l < D / 64) {
        char* params = cache.params.data + page * cache.params.page + (long long)row * cache.params.row + head * cache.params.head;
        reinterpret_cast<uint32_t*>(params)[l] = l ? pair[D / 64 - 1] : pair[0];
    }
}

template <class T, int D, int SINK>
__global__ void __launch_bounds__(kThreads, 3) gsr_rope_kernel(const __grid_constant__ RopeAppendParams a,
                                                            const __grid_constant__ RopePlan plan) {
    constexpr int LANES = D / 16, ROWS = 32 / LANES, STEPS = 4;      // rows at once, rows a lane has in flight
    const RopeParams& p = a.f;
    const int unit = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31, l = lane % LANES;
    if (unit >= plan.units) return;
    const int token = plan.by_unit(unit);
    int block = unit - token * (int)plan.by_unit.d;
    const bool is_q = block < plan.q_blocks;
    if (!is_q) block -= plan.q_blocks;
    const bool is_v = SINK != kSinkRows && !is_q && block >= plan.k_blocks;
    if (is_v) block -= plan.k_blocks;
    const int b = plan.by_seq(token), s = token - b * p.S;
    const Strided& src = is_q ? p.Q : is_v ? a.V : p.K;
    const int heads = is_q ? p.Hq : p.Hkv, h0 = block * plan.per + lane / LANES, end = min(heads, (block + 1) * plan.per);
    const LanePart at = lane_part(l, is_v || !p.table ? 0 : p.R, p.interleaved);

    uint4 raw[STEPS][2];
    const T* from = static_cast<const T*>(src.data) + b * src.batch + s * src.row;
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
        if (h0 + i * ROWS < end) load_part(from + (h0 + i * ROWS) * src.head, at, raw[i][0], raw[i][1]);

    int pos = s;
    if (p.table && p.positions) pos = __ldg(p.positions + token);
    const bool to_cache = SINK != kSinkRows && !is_q;
    long long page = 0;
    int row = 0;
    if (to_cache) {
        const int slot = __ldg(a.slots + token);
        if (slot < 0 || slot >= (long long)a.num_pages * a.page || (p.table && pos < 0)) return;      // padding
        page = plan.by_page(slot);
        row = slot - (int)page * a.page;
    }
    const bool known = !p.table || (pos >= 0 && pos < p.rows);
    const float* cosines = p.table + (known ? (long long)pos * p.R + 8 * l : 0);
    const T* w = static_cast<const T*>(is_q ? p.q_weight : is_v ? nullptr : p.k_weight);

#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int h = h0 + i * ROWS;
        const bool live = h < end;
        if (!__any_sync(0xffffffffu, live)) break;
        float v[16];
        if (!live) raw[i][0] = raw[i][1] = make_uint4(0u, 0u, 0u, 0u);
        unpack8<T>(raw[i][0], v);
        unpack8<T>(raw[i][1], v + 8);
        if (w) {
            float sum = 0.0f;
#pragma unroll
            for (int k = 0; k < 16; ++k) sum = fmaf(v[k], v[k], sum);
            const float r = rsqrtf(row_sum<LANES>(sum) * (1.0f / D) + p.eps);
            float weight[16];
            load_weight(w, at, weight);
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = v[k] * r * weight[k];
        }
        if (at.turns && known) rotate(v, cosines, p.R, p.interleaved, 1.0f);
        if (!known && !is_v) {
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = pos < 0 ? 0.0f : NAN;
        }
        if (SINK == kSinkRows || is_q) {
            const Strided& to = is_q ? p.Qo : p.Ko;
            if (live) store_part(static_cast<T*>(to.data) + b * to.batch + s * to.row + h * to.head, at, v);
        } else if (SINK == kSinkCache16) {
            const Strided& to = is_v ? a.Vc : a.Kc;
            if (live) store_part(static_cast<T*>(to.data) + page * to.batch + row * to.row + h * to.head, at, v);
        } else {
            store_row4<T, D>(is_v ? a.V4 : a.K4, page, row, h, at, l, live, v);
        }
    }
}

// Heads a unit takes: as many as a warp has in flight, or one step of rows where that leaves SMs without a warp.
int rope_unit_heads(long long tokens, int heads, int D, int sms) {
    const int step = 512 / D;
    return tokens * ((heads + 4 * step - 1) / (4 * step)) >= 8ll * sms ? 4 * step : step;
}

template <class T, int D, int SINK>
cudaError_t launch_rope(const RopeAppendParams& a, int sms, cudaStream_t stream) {
    const RopeParams& p = a.f;
    const long long tokens = (long long)p.B * p.S;
    RopePlan plan{Divider(1), Divider((uint32_t)p.S), Divider((uint32_t)(a.page > 0 ? a.page : 1)), 0, 0, 0, 0};
    plan.per = rope_unit_heads(tokens, p.Hq + (SINK == kSinkRows ? 1 : 2) * p.Hkv, D, sms);
    plan.q_blocks = (p.Hq + plan.per - 1) / plan.per;
    plan.k_blocks = (p.Hkv + plan.per - 1) / plan.per;
    const int blocks = plan.q_blocks + (SINK == kSinkRows ? 1 : 2) * plan.k_blocks;
    plan.by_unit = Divider((uint32_t)blocks);
    plan.units = (int)(tokens * blocks);
    gsr_rope_kernel<T, D, SINK><<<(unsigned)((plan.units + kWarps - 1) / kWarps), kThreads, 0, stream>>>(a, plan);
    return cudaGetLastError();
}
template <int SINK>
cudaError_t launch_rope_type(const RopeAppendParams& a, bool bf16, int sms, cudaStream_t stream) {
    if (a.f.D == 64)
        return bf16 ? launch_rope<__nv_bfloat16, 64, SINK>(a, sms, stream) : launch_rope<__half, 64, SINK>(a, sms, stream);
    return bf16 ? launch_rope<__nv_bfloat16, 128, SINK>(a, sms, stream) : launch_rope<__half, 128, SINK>(a, sms, stream);
}

// ---------------------------------------------------------------------------
// Gradient
// ---------------------------------------------------------------------------
// With dy the incoming gradient turned back, n = x r, dn = dy w:
//   dw = sum over rows of dy n,   dx = r (dn - n mean(dn n)) = r dn - x r^3 sum(dn x) / D.
// r is computed again from x, which has to be read anyway, so the forward pass stores nothing.  A CTA sums dw
// over its rows in registers (fp32, a lane's 16 columns), then over its warps; a second launch adds the CTAs'
// sums in their order, so that results repeat.
struct RopeBwdPlan {
    Divider by_q, by_k, by_seq;
    int q_units, k_units;               // steps of as many rows as a warp holds at once
};

template <class T, int D>
__global__ void __launch_bounds__(kThreads, 2) gsr_rope_bwd_kernel(const __grid_constant__ RopeBwdParams a,
                                                                   const __grid_constant__ RopeBwdPlan plan) {
    constexpr int LANES = D / 16, ROWS = 32 / LANES;
    __shared__ float sums[kWarps][D];
    const RopeParams& p = a.f;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LANES;
    const LanePart at = lane_part(l, p.table ? p.R : 0, p.interleaved);
#pragma unroll 1
    for (int part = 0; part < 2; ++part) {
        const Strided &G = part ? p.Ko : p.Qo, &X = part ? p.K : p.Q, &dX = part ? a.dK : a.dQ;
        const T* w = static_cast<const T*>(part ? p.k_weight : p.q_weight);
        const int units = part ? plan.k_units : plan.q_units, heads = part ? p.Hkv : p.Hq;
        const Divider& by = part ? plan.by_k : plan.by_q;
        float dw[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) dw[k] = 0.0f;
        // a step's rows are loaded before the arithmetic of the step before it
        struct Rows {
            uint4 g[2], x[2];
            long long to;               // where this lane's row of dX starts
            int pos;
            bool live;
        };
        auto load = [&](int unit, Rows& r) {
            r.g[0] = r.g[1] = r.x[0] = r.x[1] = make_uint4(0u, 0u, 0u, 0u);
            r.live = false;
            if (unit >= units) return;
            const int token = by(unit), h = (unit - token * (int)by.d) * ROWS + lane / LANES, b = plan.by_seq(token), s = token - b * p.S;
            r.pos = p.table && p.positions ? __ldg(p.positions + token) : s;
            r.live = h < heads;
            if (!r.live) return;
            load_part(static_cast<const T*>(G.data) + b * G.batch + s * G.row + h * G.head, at, r.g[0], r.g[1]);
            if (w) load_part(static_cast<const T*>(X.data) + b * X.batch + s * X.row + h * X.head, at, r.x[0], r.x[1]);
            r.to = b * dX.batch + s * dX.row + h * dX.head;
        };
        const int first = blockIdx.x * kWarps + warp, stride = gridDim.x * kWarps;
        Rows now, next;
        load(first, now);
#pragma unroll 1
        for (int unit = first; unit < units; unit += stride) {
            load(unit + stride, next);
            const bool known = !p.table || (now.pos >= 0 && now.pos < p.rows), counts = now.live && (!p.table || now.pos >= 0);
            float dy[16];
            unpack8<T>(now.g[0], dy);
            unpack8<T>(now.g[1], dy + 8);
            if (at.turns && known) rotate(dy, p.table + (long long)now.pos * p.R + 8 * l, p.R, p.interleaved, -1.0f);
            if (!known) {
#pragma unroll
                for (int k = 0; k < 16; ++k) dy[k] = counts ? NAN : 0.0f;
            }
            if (w) {
                float v[16], weight[16];
                unpack8<T>(now.x[0], v);
                unpack8<T>(now.x[1], v + 8);
                load_weight(w, at, weight);
                float square = 0.0f, dot = 0.0f;
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    square = fmaf(v[k], v[k], square);
                    dot = fmaf(dy[k] * weight[k], v[k], dot);
                }
                const float r = rsqrtf(row_sum<LANES>(square) * (1.0f / D) + p.eps);
                const float back = row_sum<LANES>(dot) * (1.0f / D) * r * r * r;
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    if (counts) dw[k] = fmaf(dy[k] * v[k], r, dw[k]);       // padding adds nothing, whatever it holds
                    dy[k] = counts ? r * dy[k] * weight[k] - v[k] * back : 0.0f;
                }
            }
            if (now.live) store_part(static_cast<T*>(dX.data) + now.to, at, dy);
            now = next;
        }
        if (!w) continue;
#pragma unroll
        for (int k = 0; k < 16; ++k)
#pragma unroll
            for (int o = LANES; o < 32; o <<= 1) dw[k] += __shfl_xor_sync(0xffffffffu, dw[k], o);
        __syncthreads();
        if (lane < LANES) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                sums[warp][8 * at.c0 + k] = dw[k];
                sums[warp][8 * at.c1 + k] = dw[8 + k];
            }
        }
        __syncthreads();
        if (threadIdx.x < D) {
            float t = 0.0f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) t += sums[k][threadIdx.x];
            a.parts[((long long)part * a.ctas + blockIdx.x) * D + threadIdx.x] = t;
        }
    }
}

// dw = sum of the CTAs' parts, a CTA for 32 columns: 32 lanes of rows, each in ascending order.
__global__ void __launch_bounds__(1024) gsr_rope_weights_kernel(const float* parts, int ctas, int D, float* dq_weight, float* dk_weight) {
    __shared__ float sums[32][33];
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), y = threadIdx.x >> 5;
    float* to = blockIdx.y ? dk_weight : dq_weight;
    if (!to) return;
    float t = 0.0f;
#pragma unroll 8
    for (int i = y; i < ctas; i += 32) t += parts[((long long)blockIdx.y * ctas + i) * D + col];
    sums[y][threadIdx.x & 31] = t;
    __syncthreads();
    if (y == 0) {
        t = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) t += sums[i][threadIdx.x];
        to[col] = t;
    }
}

template <class T, int D>
cudaError_t launch_bwd(const RopeBwdParams& a, cudaStream_t stream) {
    const RopeParams& p = a.f;
    const long long tokens = (long long)p.B * p.S;
    cudaError_t e = cudaSuccess;
    if (a.ctas > 0) {
        RopeBwdPlan plan{Divider(1), Divider(1), Divider((uint32_t)p.S), 0, 0};
        const int step = 512 / D, q_blocks = (p.Hq + step - 1) / step, k_blocks = (p.Hkv + step - 1) / step;
        if (q_blocks) plan.by_q = Divider((uint32_t)q_blocks);
        if (k_blocks) plan.by_k = Divider((uint32_t)k_blocks);
        plan.q_units = (int)(tokens * q_blocks);
        plan.k_units = (int)(tokens * k_blocks);
        gsr_rope_bwd_kernel<T, D><<<(unsigned)a.ctas, kThreads, 0, stream>>>(a, plan);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (a.dq_weight || a.dk_weight) {
        gsr_rope_weights_kernel<<<dim3(D / 32, 2), 1024, 0, stream>>>(a.parts, a.ctas, D, a.dq_weight, a.dk_weight);
        e = cudaGetLastError();
    }
    return e;
}

// ---------------------------------------------------------------------------
// Rows of a cache of 4 bits, read back
// ---------------------------------------------------------------------------
// A lane takes 16 values: 8 bytes of codes become 32 bytes.  s x code is exact in fp32, so a value is rounded
// once there and once to T.
template <class T, int D>
__global__ void __launch_bounds__(kThreads) gsr_read4_kernel(const __grid_constant__ Read4Params p, const Divider by_head,
                                                             const Divider by_page, long long rows) {
    constexpr int LANES = D / 16, PER = kThreads / LANES;
    const long long id = (long long)blockIdx.x * PER + threadIdx.x / LANES;      // a token's heads of K, then of V
    const int l = threadIdx.x % LANES;
    if (id >= rows) return;
    const bool is_v = id >= rows / 2;
    const int r = (int)(is_v ? id - rows / 2 : id), n = by_head(r), h = r - n * p.H;
    const int slot = __ldg(p.slots + n);
    if (slot < 0 || slot >= (long long)p.num_pages * p.page) return;
    const long long page = by_page(slot);
    const int row = slot - (int)page * p.page;
    const Cache4& cache = is_v ? p.V4 : p.K4;
    const Strided& to = is_v ? p.V : p.K;
    const uint2 codes = __ldg(reinterpret_cast<const uint2*>(cache.codes.data + page * cache.codes.page +
                                                             (long long)row * cache.codes.row + h * cache.codes.head) + l);
    const float2 sm = Pair<T>::unpack(__ldg(reinterpret_cast<const uint32_t*>(cache.params.data + page * cache.params.page +
                                                                             (long long)row * cache.params.row +
                                                                             h * cache.params.head) + l / 4));
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = fmaf(sm.x, (float)((i < 8 ? codes.x : codes.y) >> (4 * (i & 7)) & 15u), sm.y);
    uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(to.data) + n * to.row + h * to.head) + 2 * l;
    out[0] = pack8<T>(v);
    out[1] = pack8<T>(v + 8);
}

template <class T, int D>
cudaError_t launch_read(const Read4Params& p, cudaStream_t stream) {
    const long long rows = 2ll * p.N * p.H;
    constexpr int PER = kThreads / (D / 16);
    gsr_read4_kernel<T, D><<<(unsigned)((rows + PER - 1) / PER), kThreads, 0, stream>>>(p, Divider((uint32_t)p.H),
                                                                                        Divider((uint32_t)p.page), rows);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_fwd(const RopeParams& p, bool bf16, int sms, cudaStream_t stream) {
    RopeAppendParams a{};
    a.f = p;
    return launch_rope_type<kSinkRows>(a, bf16, sms, stream);
}

cudaError_t launch_rope_append(const RopeAppendParams& p, bool bf16, bool four_bits, int sms, cudaStream_t stream) {
    return four_bits ? launch_rope_type<kSinkCache4>(p, bf16, sms, stream) : launch_rope_type<kSinkCache16>(p, bf16, sms, stream);
}

// CTAs of the gradient: two an SM, or fewer where there are fewer rows.
int rope_bwd_ctas(long long batch, long long heads_q, long long heads_kv, long long seq, int D, int sms) {
    const int step = 512 / D;                            // rows of a warp at once
    const double warps = (double)(batch * seq) * (double)((heads_q > heads_kv ? heads_q : heads_kv) + step - 1) / step;
    const double ctas = (warps + kWarps - 1) / kWarps;
    return ctas < 2.0 * sms ? (int)ctas : 2 * sms;
}

cudaError_t launch_rope_bwd(const RopeBwdParams& p, bool bf16, cudaStream_t stream) {
    if (p.f.D == 64) return bf16 ? launch_bwd<__nv_bfloat16, 64>(p, stream) : launch_bwd<__half, 64>(p, stream);
    return bf16 ? launch_bwd<__nv_bfloat16, 128>(p, stream) : launch_bwd<__half, 128>(p, stream);
}

cudaError_t launch_read4(const Read4Params& p, bool bf16, cudaStream_t stream) {
    if (p.D == 64) return bf16 ? launch_read<__nv_bfloat16, 64>(p, stream) : launch_read<__half, 64>(p, stream);
    return bf16 ? launch_read<__nv_bfloat16, 128>(p, stream) : launch_read<__half, 128>(p, stream);
}

}  // namespace gsr
