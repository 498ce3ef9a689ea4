// verify.cu - which drafted tokens the target's probabilities keep, and the token that follows them.
//
// Node c below node n, token x, is kept where u T q(x) < r(x), its siblings before it having been refused.  r is what is
// left of the target's distribution p after n: r = p and T = 1 at first; a refusal leaves r' = max(r - T q, 0),
// T' = sum r' where q is the distribution that x was drawn from, and r without x, T' = T - r(x) where it was not drawn
// (q is 1 at x).  At the last kept node the next token is drawn from r: the first v with r(0) + .. + r(v) > u sum(r).
// Tokens kept or drawn so are distributed as the target's own.
//
// What bounds it: one row of V floats a request, two where a draft with probabilities was refused; below some MB the
// latency of three dependent reads and two cluster barriers.  A cluster of 8 CTAs shares a request's row (one CTA a
// request would read 0.5 MB alone).  Sums are of fixed-point integers, 45 bits behind the point: no order of adding
// changes them, so the row can be cut anywhere and the drawn token is the same on each run; it differs from sums
// in 64-bit floats only where u falls within about V 2^-46 of a border.
//
// Measured, captured: 64 chains of 8 nodes over 128000 tokens with draft probabilities 20.7 us (3.2 TB/s: a walk, a pass, a
// barrier, a 64th of the row again, one after another); 32 trees of 24 nodes over 49999 tokens 13.5 us; one chain over
// 32000 tokens 7.4 us, latency alone.
#include "gsr.h"
#include "serving.h"

namespace gsr {
namespace {

constexpr int kVerifyThreads = 256, kVerifyWarps = kVerifyThreads / 32, kVerifyCtas = 8, kVerifyAtOnce = 8;
constexpr int kMaxNodes = GSR_TREE_MAX_NODES;
static_assert(kMaxNodes == 64, "a warp holds two nodes a lane");

enum Step : int { kStepNone, kStepSum, kStepDraw };

// What a request's first CTA asks of all of them: sum (and draw from) what is left of a row.
struct Order {
    int step, refused;
    int row;                        // of the target, the last kept node's
    int with_draft;
    int what[kMaxNodes];            // refused drafts: their rows, or without probabilities their tokens
    double total[kMaxNodes];        // T before each refusal
};

__device__ __forceinline__ uint32_t smem_of(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ uint32_t of_cta(uint32_t addr, int rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    return a;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Probabilities as the sums count them: NaN is 0, the rest cut to 0..1.
__device__ __forceinline__ float sane(float p) { return fminf(fmaxf(p, 0.0f), 1.0f); }
// p in units of 2^-45, hi 2^23 + lo: two sums with a constant round p to 2^-22 and what is left to 2^-45 and leave the integers in
// their low bits (a conversion to 64 bits costs four times as much).  Larger p, larger or equal result.
struct Fixed {
    int hi, lo;
};
__device__ __forceinline__ Fixed fixed(float p) {
    const float x = sane(p), a = __fadd_rn(x, 2.0f);                       // 2..3: steps of 2^-22
    const float rest = __fsub_rn(x, __fsub_rn(a, 2.0f));                   // exact, at most 2^-23
    const float b = __fadd_rn(rest, 0x1.8p-22f);                           // 2^-22..2^-21: steps of 2^-45
    return {__float_as_int(a) - __float_as_int(2.0f), __float_as_int(b) - __float_as_int(0x1.8p-22f)};
}
__device__ __forceinline__ long long whole(Fixed f) { return (long long)f.hi * (1 << 23) + f.lo; }
constexpr double kOne = 35184372088832.0;           // 2^45
__device__ __forceinline__ unsigned long long warp_total(unsigned long long x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// What is left of the target's row.
struct Left {
    const float* target;
    const float* draft;
    long long draft_row;
    const Order* order;
    int refused;
    bool two;                                       // the first refused draft's row goes off the target's
    const float* first;
    // at column v
    __device__ __forceinline__ long long at(int v, float p, float q) const {
        long long r = whole(fixed(p));
        if (!two) {
            for (int i = 0; i < refused; ++i)
                if (order->what[i] == v) r = 0;
            return r;
        }
        r = max(r - whole(fixed(q)), 0ll);
        for (int i = 1; i < refused; ++i) {
            const double less = order->total[i] * (double)whole(fixed(__ldg(draft + order->what[i] * draft_row + v)));
            r = max(r - __double2ll_rn(less), 0ll);
        }
        return r;
    }
    // a lane's columns v0, v0 + 32, ..: their sum, and each one in x where it is asked for
    template <bool KEEP>
    __device__ __forceinline__ long long some(int v0, int hi, long long (&x)[kVerifyAtOnce]) const {
        float p[kVerifyAtOnce], q[kVerifyAtOnce];
#pragma unroll
        for (int k = 0; k < kVerifyAtOnce; ++k) {
            const int v = v0 + 32 * k;
            p[k] = v < hi ? __ldg(target + v) : 0.0f;
            q[k] = two && v < hi ? __ldg(first + v) : 0.0f;
        }
        if (!KEEP && (!two || refused == 1)) {      // nothing but max(p - q, 0)
            int hi_sum = 0, lo_sum = 0;
#pragma unroll
            for (int k = 0; k < kVerifyAtOnce; ++k) {
                const Fixed a = fixed(p[k]), b = fixed(q[k]);
                if (sane(p[k]) > sane(q[k])) {
                    hi_sum += a.hi - b.hi;
                    lo_sum += a.lo - b.lo;
                }
            }
            return (long long)hi_sum * (1 << 23) + lo_sum;
        }
        long long total = 0;
#pragma unroll
        for (int k = 0; k < kVerifyAtOnce; ++k) {
            const long long r = v0 + 32 * k < hi ? at(v0 + 32 * k, p[k], q[k]) : 0;
            if (KEEP) x[k] = r;
            total += r;
        }
        return total;
    }
    // the sum over columns [lo, hi), by a warp
    __device__ __forceinline__ unsigned long long sum(int lo, int hi, int lane) const {
        long long total = 0, x[kVerifyAtOnce];
        for (int v0 = lo + lane; v0 < hi; v0 += 32 * kVerifyAtOnce) total += some<false>(v0, hi, x);
        if (!two)                                   // less the refused tokens, each of them once in the list
            for (int i = lane; i < refused; i += 32) {
                const int v = order->what[i];
                if (v >= lo && v < hi) total -= whole(fixed(__ldg(target + v)));
            }
        return warp_total((unsigned long long)total);
    }
};

__global__ void __cluster_dims__(kVerifyCtas, 1, 1) __launch_bounds__(kVerifyThreads, 4)
    gsr_verify_kernel(const __grid_constant__ VerifyParams p, const int seg) {
    __shared__ Order s_order, s_own;                 // the request's (in its first CTA), and this CTA's copy
    __shared__ unsigned long long s_totals[kVerifyCtas], s_warps[kVerifyWarps];
    const int rank = blockIdx.x % kVerifyCtas, b = blockIdx.x / kVerifyCtas;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool leads = rank == 0 && warp == 0;

    // ---- the walk down the tree, by the first CTA's first warp: lane i holds nodes i and i + 32
    int nodes = 0, q0 = 0, cur = 0, next = 1, kept = 0, refused = 0, parent[2], token[2];
    float u[2], pt[2], qt[2];
    bool gone[2] = {false, false};                   // refused below `cur`
    double left = 1.0;                               // T
    if (leads) {
        q0 = __ldg(p.q_starts + b);
        nodes = q0 < 0 ? 0 : min(min(__ldg(p.q_starts + b + 1) - q0, p.max_nodes), p.N - q0);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int c = lane + 32 * k;
            parent[k] = token[k] = -1;
            u[k] = pt[k] = qt[k] = 0.0f;
            if (c > 0 && c < nodes) {
                parent[k] = p.parents ? __ldg(p.parents + q0 + c) : c - 1;
                token[k] = __ldg(p.tokens + q0 + c);
                u[k] = __ldg(p.u_accept + q0 + c);
                if (parent[k] >= 0 && parent[k] < c && token[k] >= 0 && token[k] < p.V) {
                    pt[k] = sane(__ldg(p.target + (q0 + parent[k]) * p.target_row + token[k]));
                    if (p.draft) qt[k] = sane(__ldg(p.draft + (q0 + c) * p.draft_row + token[k]));
                }
                if (!(u[k] > 0.0f)) u[k] = 0.0f;
            }
        }
    }
    bool have_total = true;                          // `left` is up to date

    for (;;) {
        if (leads) {
            int step = nodes > 0 ? kStepDraw : kStepNone;
            while (step == kStepDraw) {
                const uint32_t lo = __ballot_sync(0xffffffffu, parent[0] == cur && lane >= next);
                const uint32_t hi = __ballot_sync(0xffffffffu, parent[1] == cur && lane + 32 >= next);
                if (!(lo | hi)) break;
                const int c = lo ? __ffs(lo) - 1 : 31 + __ffs(hi), from = c & 31;
                const int x = __shfl_sync(0xffffffffu, c < 32 ? token[0] : token[1], from);
                const double uc = __shfl_sync(0xffffffffu, c < 32 ? u[0] : u[1], from);
                double r = __shfl_sync(0xffffffffu, c < 32 ? pt[0] : pt[1], from);
                double q = __shfl_sync(0xffffffffu, c < 32 ? qt[0] : qt[1], from);
                if (!p.draft) {
                    q = 1.0;
                    if (__any_sync(0xffffffffu, (gone[0] && token[0] == x) || (gone[1] && token[1] == x))) r = 0.0;
                } else if (refused > 0) {
                    if (!have_total) {               // ask for the sum first
                        step = kStepSum;
                        break;
                    }
                    for (int i = 0; i < refused; ++i) {
                        const float y = x >= 0 && x < p.V ? __ldg(p.draft + s_order.what[i] * p.draft_row + x) : 0.0f;
                        r = fmax(r - s_order.total[i] * (double)sane(y), 0.0);
                    }
                }
                next = c + 1;
                if (uc * left * q < r) {
                    if (lane == 0) p.path[(long long)b * p.max_nodes + kept] = c;
                    ++kept;
                    cur = c;
                    refused = 0;
                    left = 1.0;
                    have_total = true;
                    gone[0] = gone[1] = false;
                } else {
                    // without probabilities a token is listed once
                    if (p.draft || r > 0.0) {
                        if (lane == 0) {
                            s_order.what[refused] = p.draft ? q0 + c : x;
                            s_order.total[refused] = left;
                        }
                        __syncwarp();
                        ++refused;
                    }
                    if (p.draft) have_total = false;
                    else left -= r;
                    if (lane == from) gone[c >> 5] = true;
                }
            }
            if (lane == 0) {
                s_order.step = step;
                s_order.refused = refused;
                s_order.row = q0 + cur;
                s_order.with_draft = p.draft != nullptr;
            }
            __syncwarp();
        }
        cluster_sync();
        {   // the order, from the first CTA
            const uint32_t from = of_cta(smem_of(&s_order), 0);
            uint32_t* to = reinterpret_cast<uint32_t*>(&s_own);
            for (int i = threadIdx.x; i < (int)(sizeof(Order) / 4); i += kVerifyThreads) {
                uint32_t x;
                asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(x) : "r"(from + 4 * i) : "memory");
                to[i] = x;
            }
        }
        __syncthreads();
        const bool two = s_own.refused > 0 && s_own.with_draft;
        const Left rest{p.target + s_own.row * p.target_row, p.draft, p.draft_row, &s_own, s_own.refused, two,
                        two ? p.draft + s_own.what[0] * p.draft_row : nullptr};
        const int lo = min((long long)(rank * kVerifyWarps + warp) * seg, (long long)p.V), hi = min((long long)lo + seg, (long long)p.V);
        unsigned long long mine = 0;
        if (s_own.step != kStepNone) mine = rest.sum(lo, hi, lane);
        if (lane == 0) s_warps[warp] = mine;
        __syncthreads();
        if (threadIdx.x < kVerifyCtas) {
            unsigned long long t = 0;
#pragma unroll
            for (int i = 0; i < kVerifyWarps; ++i) t += s_warps[i];
            asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(of_cta(smem_of(&s_totals[rank]), threadIdx.x)), "l"(t) : "memory");
        }
        cluster_sync();                              // after it no CTA reaches into another
        unsigned long long total = 0, before = 0;
#pragma unroll
        for (int i = 0; i < kVerifyCtas; ++i) {
            if (i < rank) before += s_totals[i];
            total += s_totals[i];
        }
        if (s_own.step == kStepSum) {
            left = (double)total / kOne;
            have_total = true;
            continue;
        }
        if (s_own.step == kStepDraw && total == 0 && s_own.refused > 0) {
            // nothing is left (the refusal was a rounding's): draw from the target's own row
            refused = 0;
            next = nodes;
            continue;
        }
        if (leads) {
            for (int i = kept + lane; i < p.max_nodes; i += 32) p.path[(long long)b * p.max_nodes + i] = -1;
            if (lane == 0) {
                p.counts[b] = kept;
                if (total == 0) p.next[b] = -1;
            }
        }
        if (s_own.step == kStepNone || total == 0) return;
        // ---- the first column whose running sum exceeds u total: this CTA's, a warp's part, an eighth of it
        const float us = __ldg(p.u_sample + b);
        unsigned long long at = us > 0.0f ? (us < 1.0f ? __double2ull_rd((double)us * (double)total) : total - 1) : 0;
        if (at >= total) at = total - 1;
        if (at < before || at - before >= s_totals[rank]) return;
        at -= before;
        int part = 0;
        while (part < kVerifyWarps - 1 && at >= s_warps[part]) at -= s_warps[part++];
        __syncthreads();
        const int start = min((long long)(rank * kVerifyWarps + part) * seg, (long long)p.V), stop = min((long long)start + seg, (long long)p.V);
        const int eighth = seg / kVerifyWarps, a0 = min(start + warp * eighth, stop), a1 = min(a0 + eighth, stop);
        long long x[kVerifyAtOnce];                  // where an eighth is a lane's eight columns, they are kept
        const bool keep = eighth <= 32 * kVerifyAtOnce;
        const unsigned long long piece = keep ? warp_total((unsigned long long)rest.some<true>(a0 + lane, a1, x)) : rest.sum(a0, a1, lane);
        if (lane == 0) s_warps[warp] = piece;
        __syncthreads();
        part = 0;
        while (part < kVerifyWarps - 1 && at >= s_warps[part]) at -= s_warps[part++];
        if (warp != part) return;
        for (int v0 = a0; v0 < a1; v0 += 32 * kVerifyAtOnce) {
            if (!keep) rest.some<true>(v0 + lane, a1, x);
#pragma unroll
            for (int k = 0; k < kVerifyAtOnce; ++k) {
                unsigned long long run = (unsigned long long)x[k];
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const unsigned long long y = __shfl_up_sync(0xffffffffu, run, o);
                    if (lane >= o) run += y;
                }
                const uint32_t past = __ballot_sync(0xffffffffu, run > at);
                if (past) {
                    if (lane == 0) p.next[b] = v0 + 32 * k + __ffs(past) - 1;
                    return;
                }
                at -= __shfl_sync(0xffffffffu, run, 31);
            }
        }
        return;
    }
}

}  // namespace

cudaError_t launch_verify(const VerifyParams& p, cudaStream_t stream) {
    // a warp's part of a row: whole loads of a warp for each eighth
    const int unit = 32 * kVerifyWarps, parts = kVerifyCtas * kVerifyWarps;
    const int seg = (int)((((long long)p.V + parts - 1) / parts + unit - 1) / unit * unit);
    gsr_verify_kernel<<<(unsigned)(p.B * kVerifyCtas), kVerifyThreads, 0, stream>>>(p, seg);
    return cudaGetLastError();
}

}  // namespace gsr
