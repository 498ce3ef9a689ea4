// attention_masked_fwd.cuh - attention forward with a document or prefix mask, capped scores, a
// distance bias and grouped heads:  O = softmax(score(Q K^T)) V.  Instantiated per element type.
//
// Every mask here leaves a query one interval of keys [lo, hi), and intervals never step back from
// one query to the next (row_interval), so a block of queries reads the key tiles from its first
// row's lo to its last row's hi and skips the rest: a packed row of documents costs what its
// documents cost, whatever the row's length.
//
//  * one CTA per SM, 384 threads: warp 0 takes work items and issues TMA copies, one lane of warp 1
//    issues every MMA, warps 4-7 run the softmax of query tile 0 and warps 8-11 that of tile 1, one
//    thread per query row (= TMEM lane).  A work item is two 128-query tiles of one head;
//  * items are CTAs of the grid that a running CTA takes over by cluster launch control: the
//    hardware keeps the count, so nothing in memory is shared between launches, captured ones too;
//  * per query tile, S(t) = Q K_t^T lands in 128 TMEM columns, the softmax writes P(t) over the
//    last 64 of them, and O += P(t) V_t reads P from TMEM.  The two tiles alternate on the tensor
//    core: while one is exponentiated, the other's products run;
//  * the exponent base moves only when a tile's maximum exceeds it by more than 2^8, so P <= 256
//    and O is rarely rescaled.  P is rounded to the operands' type for the second product (the
//    tensor core takes both operands in one type); its sum l is kept in fp32 from unrounded values;
//  * where items are few for the SMs, their key tiles are cut into p.splits runs, each an item that
//    leaves its part (maximum, sum, O in fp32) in the workspace, and a second launch joins them.
//
// Masked scores are replaced by -inf, so what K holds there is never used.  A masked V row enters
// the product as 0 V, which is NaN where V is not finite.  Only edge tiles, those that not all rows of the item
// see whole, have masked rows.  An item with a row that is not finite, and with something in the V of its edge
// tiles that is not finite either, goes on a list, and after its last item the CTA runs those of the list again
// with edge tiles cleaned before they are handed on ("Infinities and NaN behind a mask" in attention_common.cuh).
// A CTA whose list is full takes over no further CTA; those left start in its place.  The second run is a copy of
// the code of its own: what the first one would need for it in its loops costs 2 to 9 %, and cleaning every edge
// tile at once, which needs no second run, 5 to 15 %, since V lands late in an item's last tiles.
#pragma once

#include <atomic>
#include <type_traits>

#include "attention_common.cuh"
#include "ptx_attention.cuh"

namespace gsr {

template <class T_, int D_, int MODE_>
struct MaskedFwdCfg {
    using T = T_;
    static constexpr int D = D_;
    static constexpr int MODE = MODE_;
    static constexpr int BQ = 128, BKV = 128;
    static constexpr int NQ = 2;
    static constexpr int DCH = D / 64;                // 64-column (128-byte) chunks per row
    static constexpr int CHUNK_BYTES = 128 * 128;
    static constexpr int Q_BYTES = BQ * D * 2;
    static constexpr int KV_BYTES = BKV * D * 2;
    static constexpr int SM_THREADS = 128 * NQ;
    static constexpr int NUM_THREADS = 128 + SM_THREADS;
    // 384 threads start with 168 registers each; the copying and issuing warps' group gives some to
    // the softmax groups, whose threads hold a row of 128 scores: 72 + 2 x 216 = 3 x 168
    static constexpr int CONTROL_REGS = 72, SOFTMAX_REGS = 216;
    static constexpr int QBUF = D == 64 ? 2 : 1;      // Q sets that fit: with two, the next item's loads early
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = OFF_Q + QBUF * NQ * Q_BYTES;   // ring of 2 entries {K_t, V_(t-1)}
    static constexpr int OFF_V = OFF_K + 2 * KV_BYTES;
    static constexpr int OFF_BAR = OFF_V + 2 * KV_BYTES;
    static constexpr int NUM_BARS = 22;
    static constexpr int OFF_CLC = OFF_BAR + NUM_BARS * 8;      // 16-byte aligned
    static constexpr int OFF_ITEM = OFF_CLC + 16;               // 2 x 12 ints
    static constexpr int AGAIN = 30;                            // items to run again
    static constexpr int OFF_AGAIN = OFF_ITEM + 96;             // their count, the last four that went there, 3 words each
    static constexpr int OFF_BAR_AGAIN = OFF_AGAIN + 24 + AGAIN * 12;   // the second run's barriers
    static constexpr int OFF_MISC = OFF_BAR_AGAIN + NUM_BARS * 8;
    static constexpr int SMEM_BYTES = OFF_MISC + 16;
    static constexpr int TMEM_COLS = 512;
    static constexpr uint32_t T_S = 0, T_O = 256, P_COL = 64;
    static constexpr uint32_t IDESC_S = idesc_16_f32(Elem<T>::bf16, BQ, BKV, false, false);
    static constexpr uint32_t IDESC_PV = idesc_16_f32(Elem<T>::bf16, BQ, D, false, true);
    static constexpr float RESCALE_LOG2 = 8.0f;
    static_assert(D == 64 || D == 128, "head_dim 64 or 128");
    static_assert(SMEM_BYTES <= 232448 && OFF_CLC % 16 == 0, "shared memory");
    static_assert(T_O + NQ * D <= TMEM_COLS, "TMEM budget");
};

// Part `split` of a row in the workspace.
__device__ __forceinline__ long long part_index(const MaskedFwdParams& p, int b, int h, int split, int i) {
    return (((long long)b * p.mask.Hq + h) * p.splits + split) * p.mask.Sq + i;
}

// The keys that every row of an item (two query tiles) with keys sees; a row without any among them leaves none.
// Lane 2q brings lo and hi of tile q's first row, lane 2q + 1 of its last.
struct Common {
    int lo, hi;
    // Whether not all rows see the key tile whole.
    __device__ __forceinline__ bool edge(int key_tile) const { return key_tile * 128 < lo || (key_tile + 1) * 128 > hi; }
};
__device__ __forceinline__ Common common_keys(int lo, int hi) {
    Common c{0, INT_MAX};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int first_lo = __shfl_sync(0xffffffffu, lo, 2 * q), first_hi = __shfl_sync(0xffffffffu, hi, 2 * q);
        const int last_lo = __shfl_sync(0xffffffffu, lo, 2 * q + 1), last_hi = __shfl_sync(0xffffffffu, hi, 2 * q + 1);
        if (first_lo < last_hi) {
            c.lo = max(c.lo, last_lo);
            c.hi = min(c.hi, first_hi);
        }
    }
    return c;
}
// The interval that lane `lane` of an item brings there (empty outside [0, Sq)).
__device__ __forceinline__ void item_interval(const MaskArgs& mk, int b, int q_base, int lane, int& lo, int& hi) {
    lo = hi = 0;
    const int first = q_base + (lane >> 1 & 1) * 128;
    const int row = lane & 1 ? min(first + 128, mk.Sq) - 1 : first;
    if (lane < 4 && first < mk.Sq) row_interval(mk, b, row, lo, hi);
}

// A softmax warp's rows of item n are written.  In the second run (SECOND) they get what they still lack: the columns
// that V cleaned from edge tiles makes infinite or NaN.  In the first one of them is not finite, and the item goes
// on the list if the V of its edge tiles is not finite either.
template <class Cfg, bool SECOND>
__device__ __noinline__ void after_item(const MaskedFwdParams& p, uint32_t n, int b, int h, int q_base, int split) {
    using T = typename Cfg::T;
    constexpr int D = Cfg::D;
    extern __shared__ __align__(1024) uint8_t smem[];
    const MaskArgs& mk = p.mask;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = (warp - 4) >> 2;
    const int qi = q_base + q * 128 + (warp & 3) * 32 + lane;
    int lo, hi;
    item_interval(mk, b, q_base, lane, lo, hi);
    const Common common = common_keys(lo, hi);
    const int k0 = __shfl_sync(0xffffffffu, lo, 2 * q) / 128, k1 = (__shfl_sync(0xffffffffu, hi, 2 * q + 1) + 127) / 128;
    const T* v = static_cast<const T*>(p.V.data) + b * p.V.batch + h / mk.group * p.V.head;
    lo = hi = 0;
    if (qi < mk.Sq) row_interval(mk, b, qi, lo, hi);
    for (int k = k0; k < k1; ++k) {
        if (!common.edge(k)) continue;
        const int end = min((k + 1) * 128, mk.Skv);
        if constexpr (SECOND) {
            if (p.splits > 1)
                spread_not_finite<T, D, false>(v, p.V.row, k * 128, end, lo, hi, p.parts + part_index(p, b, h, split, qi) * D,
                                               qi < mk.Sq, lane);
            else
                spread_not_finite<T, D, false>(v, p.V.row, k * 128, end, lo, hi,
                                               static_cast<uint16_t*>(p.O.data) + b * p.O.batch + h * p.O.head + (long long)qi * p.O.row,
                                               qi < mk.Sq, lane);
        } else {
            if (rows_not_finite<T, D>(v, p.V.row, k * 128, end, lane)) {
                // words: the count, then where item n puts n (n + 4 is published once every softmax warp is past n), the list
                uint32_t* words = reinterpret_cast<uint32_t*>(smem + Cfg::OFF_AGAIN);
                if (lane == 0 && atomicExch(words + 1 + (n & 3u), n) != n) {
                    uint32_t* to = words + 6 + 3 * atomicAdd(words, 1u);
                    to[0] = b * mk.Hq + h;
                    to[1] = q_base;
                    to[2] = split;
                }
                break;
            }
        }
    }
    __syncwarp();
}

// This thread's row of a part (`real`), the accumulator from TMEM column `col` on if there were steps; true if it is
// not finite.  Kept out of the kernel's own code, whose runs without parts it made 1 to 2 % slower.
template <int D>
__device__ __noinline__ bool store_part(const MaskedFwdParams& p, long long part, bool steps, bool real, uint32_t col, float m,
                                        float l) {
    float z0 = 0.0f, z1 = 0.0f;                          // 0 x, NaN where x is not finite
    if (steps) {
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
            uint32_t rr[32];
            __syncwarp();
            tmem_ld_32x32b_x32(col + c * 32, rr);
            tmem_ld_wait(rr);
#pragma unroll
            for (int i = 0; i < 32; i += 2) ffma2(z0, z1, __uint_as_float(rr[i]), __uint_as_float(rr[i + 1]), 0.0f, 0.0f, z0, z1);
            if (real)
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                    *reinterpret_cast<uint4*>(p.parts + part * D + c * 32 + i) = make_uint4(rr[i], rr[i + 1], rr[i + 2], rr[i + 3]);
        }
    }
    if (real) p.parts_ml[part] = make_float2(m, l);
    tcgen05_fence_before();
    return z0 + z1 != 0.0f;
}

// Rows from their parts, one warp each, in the parts' order; lane s holds the factor of part s.
template <class T, int D>
__global__ void __launch_bounds__(256) gsr_masked_fwd_join_kernel(const __grid_constant__ MaskedFwdParams p) {
    using V = typename std::conditional<D == 128, float4, float2>::type;
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    grid_wait();                                         // the parts' launch has finished
    if (row >= (long long)p.mask.B * p.mask.Hq * p.mask.Sq) return;
    const int i = (int)(row % p.mask.Sq), bh = (int)(row / p.mask.Sq), b = bh / p.mask.Hq, h = bh - b * p.mask.Hq;
    float2 ml = make_float2(-INFINITY, 0.0f);
    if (lane < p.splits) ml = p.parts_ml[part_index(p, b, h, lane, i)];
    float m = ml.x;
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float f = m == -INFINITY ? 0.0f : ex2_approx(ml.x - m);
    const float l = warp_sum(f == 0.0f && ml.y == ml.y ? 0.0f : ml.y * f);
    const float factor = ml.x == -INFINITY ? -1.0f : f;  // below 0: a part without keys that the row sees
    float acc[D / 32] = {};
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s) {
        const float fs = __shfl_sync(0xffffffffu, factor, s);
        if (fs < 0.0f) continue;                         // may hold anything
        const V x = *(reinterpret_cast<const V*>(p.parts + part_index(p, b, h, s, i) * D) + lane);
#pragma unroll
        for (int e = 0; e < D / 32; ++e) acc[e] = fmaf(reinterpret_cast<const float*>(&x)[e], fs, acc[e]);
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) acc[e] *= inv;
    store_row<T, D>(static_cast<T*>(p.O.data) + b * p.O.batch + h * p.O.head + (long long)i * p.O.row, lane, acc);
    if (p.lse && lane == 0) p.lse[row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// No keys at all: O = 0, lse = -inf.  One warp per row.
template <class T, int D>
__global__ void __launch_bounds__(256) gsr_masked_empty_kernel(const MaskedFwdParams p) {
    const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= (long long)p.mask.B * p.mask.Hq * p.mask.Sq) return;
    const int i = (int)(row % p.mask.Sq), bh = (int)(row / p.mask.Sq);
    const float zero[D / 32] = {};
    store_row<T, D>(static_cast<T*>(p.O.data) + (bh / p.mask.Hq) * p.O.batch + (bh % p.mask.Hq) * p.O.head + i * p.O.row,
                    threadIdx.x & 31, zero);
    if (p.lse && (threadIdx.x & 31) == 0) p.lse[row] = -INFINITY;
}

// The barriers of one run, from shared address `at` on.
struct FwdBars {
    uint32_t at;
    __device__ __forceinline__ uint32_t bar(int i) const { return at + 8u * i; }
    __device__ __forceinline__ uint32_t full(int s) const { return bar(0 + s); }
    __device__ __forceinline__ uint32_t empty(int s) const { return bar(2 + s); }
    __device__ __forceinline__ uint32_t sfull(int q) const { return bar(4 + q); }
    __device__ __forceinline__ uint32_t pfull(int q) const { return bar(6 + q); }
    __device__ __forceinline__ uint32_t odone(int q) const { return bar(8 + q); }
    __device__ __forceinline__ uint32_t item_pub(int i) const { return bar(10 + i); }
    __device__ __forceinline__ uint32_t item_read(int i) const { return bar(12 + i); }
    __device__ __forceinline__ uint32_t qfull(int b) const { return bar(14 + b); }
    __device__ __forceinline__ uint32_t qfree(int b) const { return bar(16 + b); }
    __device__ __forceinline__ uint32_t clc() const { return bar(18); }
    __device__ __forceinline__ uint32_t drain() const { return bar(19); }
    __device__ __forceinline__ uint32_t landed() const { return bar(20); }       // a ring entry that is cleaned before it is full
    // by one thread
    __device__ __forceinline__ void init(int softmax_warps) const {
        for (int s = 0; s < 2; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
            mbar_init(sfull(s), 1);
            mbar_init(pfull(s), 128);
            mbar_init(odone(s), 1);
            mbar_init(item_pub(s), 1);
            mbar_init(item_read(s), 1 + softmax_warps);          // the MMA lane and every softmax warp
            mbar_init(qfull(s), 1);
            mbar_init(qfree(s), 1);
        }
        mbar_init(clc(), 1);
        mbar_init(drain(), 1);
        mbar_init(landed(), 1);
        fence_mbarrier_init();
    }
};

template <class Cfg>
__global__ void __launch_bounds__(Cfg::NUM_THREADS, 1)
    gsr_masked_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV, const __grid_constant__ MaskedFwdParams p) {
    using T = typename Cfg::T;
    constexpr int D = Cfg::D;
    constexpr int NQ = Cfg::NQ;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023u) {                    // the 128-byte-swizzled operands need it
        if (threadIdx.x == 0) atomicCAS(p.err, 0, kDevErrKernelMaskedFwd | kDevErrLayout);
        return;
    }
    const uint32_t sb = smem_u32(smem);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::OFF_MISC);
    volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + Cfg::OFF_MISC + 4);
    volatile int* item_box = reinterpret_cast<volatile int*>(smem + Cfg::OFF_ITEM);
    volatile uint32_t* again_words = reinterpret_cast<volatile uint32_t*>(smem + Cfg::OFF_AGAIN);   // after_item

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const MaskArgs& mk = p.mask;

    // What the producer publishes of an item; b < 0: no more items.  Query tile q takes steps
    // [t0[q], t1[q]) and step t reads key tile key_tile(t).  A distance bias grows towards the row's own
    // position, which under a causal mask is its last key: from the first tile on, the maximum would
    // move and O be rescaled at nearly every step, so the keys are walked backwards there (flip >= 0; 4 x
    // 32 x 4096 x 128: 489 us, forwards 541).  Without a causal mask forwards: 975 us, backwards 1014.
    struct Item {
        int b, h, q_base, t0[NQ], t1[NQ], flip, split;
        __device__ __forceinline__ int key_tile(int t) const { return kHasBias<Cfg::MODE> && flip >= 0 ? flip - t : t; }
        __device__ __forceinline__ int first() const {
            return t1[0] > t0[0] ? (t1[1] > t0[1] ? min(t0[0], t0[1]) : t0[0]) : t0[1];
        }
        __device__ __forceinline__ int last() const {
            return t1[0] > t0[0] ? (t1[1] > t0[1] ? max(t1[0], t1[1]) : t1[0]) : t1[1];
        }
    };
    auto read_item = [&](int box) {
        volatile int* v = item_box + 12 * box;
        return Item{v[0], v[1], v[2], {v[3], v[4]}, {v[5], v[6]}, v[7], v[8]};
    };

    if (threadIdx.x == 0) {
        FwdBars{sb + Cfg::OFF_BAR}.init(Cfg::SM_THREADS / 32);
        for (int i = 0; i < 5; ++i) again_words[i] = 0u;
        *abort_flag = 0u;
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), Cfg::TMEM_COLS);
        tmem_relinquish_alloc_permit();
    }
    tcgen05_fence_before();
    __syncthreads();
    tcgen05_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const Waiter w{p.err, p.timeout_ns, abort_flag, kDevErrKernelMaskedFwd};

    auto produce = [&](auto run) {
        constexpr bool SECOND = decltype(run)::value;
        const FwdBars bars{sb + (SECOND ? Cfg::OFF_BAR_AGAIN : Cfg::OFF_BAR)};
        // ------------------------------------------------------------ items + TMA producer
        // The whole warp walks the items (lanes 0-3 find the intervals of the query tiles' first
        // and last rows); lane 0 waits, publishes and copies.
        const uint64_t pol = l2_policy_evict_last();     // K and V are read by every query block
        const int n_qb = (mk.Sq + NQ * Cfg::BQ - 1) / (NQ * Cfg::BQ);
        uint32_t n_pub = 0, n_q = 0, g = 0, n_clc = 0;   // items published, Q loads, ring entries, answers
        uint32_t armed = 0, parity = 0, q_armed = 0, q_parity = 0;
        bool drop_q = !SECOND && (p.test_flags & kTestDropFirstLoad) && blockIdx.x == 0;
        bool asked = false, landing = false;
        int item = SECOND ? 0 : blockIdx.x;              // the second run: place in the list
        const int n_again = SECOND ? (int)again_words[0] : 0;
        while (true) {
            Item it{-1, 0, 0, {0, 0}, {0, 0}, -1, 0};
            Common common{0, INT_MAX};
            if (SECOND && item == n_again) item = -1;
            if (item >= 0) {
                // query blocks from the last (under a causal mask the longest) to the first, in
                // groups of heads whose K and V stay in L2 together
                const int per_group = p.head_group * n_qb * p.splits, grp = item / per_group, r_in = item - grp * per_group;
                const int gsz = min(mk.B * mk.Hq - grp * p.head_group, p.head_group);
                int bh = grp * p.head_group + r_in % gsz;
                it.split = r_in / gsz % p.splits;
                it.q_base = (n_qb - 1 - r_in / gsz / p.splits) * NQ * Cfg::BQ;
                if (SECOND) {
                    bh = (int)again_words[6 + 3 * item];
                    it.q_base = (int)again_words[6 + 3 * item + 1];
                    it.split = (int)again_words[6 + 3 * item + 2];
                }
                it.b = bh / mk.Hq;
                it.h = bh - it.b * mk.Hq;
                int lo, hi;
                item_interval(mk, it.b, it.q_base, lane, lo, hi);
                if (SECOND) common = common_keys(lo, hi);
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    const int l = __shfl_sync(0xffffffffu, lo, 2 * q), e = __shfl_sync(0xffffffffu, hi, 2 * q + 1);
                    it.t0[q] = l / Cfg::BKV;
                    it.t1[q] = e > l ? (e + Cfg::BKV - 1) / Cfg::BKV : it.t0[q];
                }
                if (kHasBias<Cfg::MODE> && mk.causal) {
                    const int both = it.first() + it.last();
                    it.flip = both - 1;
#pragma unroll
                    for (int q = 0; q < NQ; ++q) {
                        const int t0 = it.t0[q];
                        it.t0[q] = both - it.t1[q];
                        it.t1[q] = both - t0;
                    }
                }
                if (p.splits > 1) {
                    const int from = it.first(), len = it.last() - from;
                    const int begin = from + len * it.split / p.splits, end = from + len * (it.split + 1) / p.splits;
#pragma unroll
                    for (int q = 0; q < NQ; ++q) {
                        it.t0[q] = min(max(it.t0[q], begin), end);
                        it.t1[q] = min(max(it.t1[q], begin), end);
                    }
                }
            }
            const uint32_t box = n_pub & 1u;
            // the box's previous item has been read by every role
            bool ok = lane != 0 || w.wait(bars.item_read(box), ((n_pub >> 1) & 1u) ^ 1u, kDevErrProducerEmpty);
            if (!__all_sync(0xffffffffu, ok)) break;
            if (lane == 0) {
                volatile int* v = item_box + 12 * box;
                v[0] = it.b;
                v[1] = it.h;
                v[2] = it.q_base;
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    v[3 + q] = it.t0[q];
                    v[5 + q] = it.t1[q];
                }
                v[7] = it.flip;
                v[8] = it.split;
                mbar_arrive(bars.item_pub(box));              // release: the consumers read the box after
            }
            ++n_pub;
            if (item < 0) break;
            const int t_begin = it.first(), t_end = it.last(), hk = it.h / mk.group;
            if (lane == 0) {
                if (t_begin < t_end) {
                    const int qb = (int)(n_q % Cfg::QBUF);
                    if (n_q >= (uint32_t)Cfg::QBUF)
                        ok = w.wait(bars.qfree(qb), ((n_q - Cfg::QBUF) / Cfg::QBUF) & 1u, kDevErrProducerEmpty);
                    if (ok) {
                        if (drop_q) {
                            drop_q = false;              // test hook: this Q is never loaded
                        } else {
                            const uint32_t qbase = sb + Cfg::OFF_Q + qb * NQ * Cfg::Q_BYTES;
                            mbar_arrive_expect_tx(bars.qfull(qb), NQ * Cfg::Q_BYTES);
#pragma unroll
                            for (int q = 0; q < NQ; ++q)
#pragma unroll
                                for (int c = 0; c < Cfg::DCH; ++c)
                                    tma_load_4d(qbase + q * Cfg::Q_BYTES + c * Cfg::CHUNK_BYTES, &tmQ, bars.qfull(qb), c * 64,
                                                it.q_base + q * Cfg::BQ, it.h, it.b, pol);
                            q_armed |= 1u << qb;
                            q_parity = (q_parity & ~(1u << qb)) | ((n_q / Cfg::QBUF) & 1u) << qb;
                        }
                        ++n_q;
                    }
                    // entry t: K_t (t < t_end) and V_(t-1) (t > t_begin)
                    for (int t = t_begin; ok && !SECOND && t <= t_end; ++t, ++g) {
                        const int s = (int)(g & 1u);
                        const uint32_t ph = (g >> 1) & 1u;
                        if (!(ok = w.wait(bars.empty(s), ph ^ 1u, kDevErrProducerEmpty))) break;
                        const bool has_k = t < t_end, has_v = t > t_begin;
                        mbar_arrive_expect_tx(bars.full(s), (has_k ? Cfg::KV_BYTES : 0) + (has_v ? Cfg::KV_BYTES : 0));
                        if (has_k) {
#pragma unroll
                            for (int c = 0; c < Cfg::DCH; ++c)
                                tma_load_4d(sb + Cfg::OFF_K + s * Cfg::KV_BYTES + c * Cfg::CHUNK_BYTES, &tmK, bars.full(s), c * 64,
                                            it.key_tile(t) * Cfg::BKV, hk, it.b, pol);
                        }
                        if (has_v) {
#pragma unroll
                            for (int c = 0; c < Cfg::DCH; ++c)
                                tma_load_4d(sb + Cfg::OFF_V + s * Cfg::KV_BYTES + c * Cfg::CHUNK_BYTES, &tmV, bars.full(s), c * 64,
                                            it.key_tile(t - 1) * Cfg::BKV, hk, it.b, pol);
                        }
                        armed |= 1u << s;
                        parity = (parity & ~(1u << s)) | ph << s;
                    }
                }
                // the next item, asked for once this one's copies are issued: earlier, a CTA busy with a
                // long item would hold one that another could start.  None once the list may fill up with the items
                // in flight (4 at most).
                if (!SECOND && again_words[0] > Cfg::AGAIN - 4) {
                    item = -1;
                } else if (!SECOND && ok) {
                    fence_proxy_async_smem();            // the last answer has been read
                    mbar_arrive_expect_tx(bars.clc(), 16);
                    clc_try_cancel(sb + Cfg::OFF_CLC, bars.clc());
                    asked = true;
                    if ((ok = w.wait(bars.clc(), n_clc & 1u, kDevErrProducerEmpty))) {
                        asked = false;
                        item = clc_taken(sb + Cfg::OFF_CLC);
                    }
                }
            }
            if (!SECOND) ++n_clc;
            if (!__all_sync(0xffffffffu, ok)) break;
            if (SECOND) {
                // entries that land on a barrier of their own and are full once their V is clean
                for (int t = t_begin; t_begin < t_end && t <= t_end; ++t, ++g) {
                    const int s = (int)(g & 1u);
                    const uint32_t ph = (g >> 1) & 1u;
                    const bool has_k = t < t_end, has_v = t > t_begin;
                    if (lane == 0 && (ok = w.wait(bars.empty(s), ph ^ 1u, kDevErrProducerEmpty))) {
                        mbar_arrive_expect_tx(bars.landed(), (has_k ? Cfg::KV_BYTES : 0) + (has_v ? Cfg::KV_BYTES : 0));
                        for (int c = 0; c < Cfg::DCH; ++c) {
                            if (has_k)
                                tma_load_4d(sb + Cfg::OFF_K + s * Cfg::KV_BYTES + c * Cfg::CHUNK_BYTES, &tmK, bars.landed(), c * 64,
                                            it.key_tile(t) * Cfg::BKV, hk, it.b, pol);
                            if (has_v)
                                tma_load_4d(sb + Cfg::OFF_V + s * Cfg::KV_BYTES + c * Cfg::CHUNK_BYTES, &tmV, bars.landed(), c * 64,
                                            it.key_tile(t - 1) * Cfg::BKV, hk, it.b, pol);
                        }
                        landing = !(ok = w.wait(bars.landed(), g & 1u, kDevErrProducerEmpty));
                    }
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    if (has_v && common.edge(it.key_tile(t - 1)) &&
                        pieces_not_finite<T>(smem + Cfg::OFF_V + s * Cfg::KV_BYTES, Cfg::KV_BYTES / 16, lane)) {
                        zero_not_finite<T>(smem + Cfg::OFF_V + s * Cfg::KV_BYTES, Cfg::KV_BYTES / 16, lane);
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (lane == 0) mbar_arrive(bars.full(s));
                }
                if (!ok) break;
                ++item;
            } else {
                item = __shfl_sync(0xffffffffu, item, 0);
            }
        }
        // every copy and answer under way must land before the CTA may exit
        if (lane == 0) {
            if (asked) w.drain(bars.clc(), (n_clc - 1) & 1u);
            if (landing) w.drain(bars.landed(), g & 1u);
            for (int b = 0; b < Cfg::QBUF; ++b)
                if (q_armed & (1u << b)) w.drain(bars.qfull(b), (q_parity >> b) & 1u);
            for (int s = 0; s < 2; ++s)
                if (armed & (1u << s)) w.drain(bars.full(s), (parity >> s) & 1u);
        }
        __syncwarp();
    };

    auto issue = [&](auto run) {
        constexpr bool SECOND = decltype(run)::value;
        const FwdBars bars{sb + (SECOND ? Cfg::OFF_BAR_AGAIN : Cfg::OFF_BAR)};
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0) {
            uint32_t n_item = 0, n_q = 0, g = 0;
            uint32_t pv_n[NQ] = {0u, 0u};                // pfull phases waited for, per query tile
            bool ok = true;
            while (ok) {
                const uint32_t box = n_item & 1u;
                if (!w.wait(bars.item_pub(box), (n_item >> 1) & 1u, kDevErrMmaFull)) break;
                const Item it = read_item(box);
                mbar_arrive(bars.item_read(box));
                ++n_item;
                if (it.b < 0) break;
                const int t_begin = it.first(), t_end = it.last();
                if (t_begin >= t_end) continue;
                const int qb = (int)(n_q % Cfg::QBUF);
                if (!w.wait(bars.qfull(qb), (n_q / Cfg::QBUF) & 1u, kDevErrMmaFull)) break;
                ++n_q;
                tcgen05_fence_after();
                for (int t = t_begin; ok && t <= t_end; ++t, ++g) {
                    const int s = (int)(g & 1u);
                    if (!(ok = w.wait(bars.full(s), (g >> 1) & 1u, kDevErrMmaFull))) break;   // K_t and V_(t-1)
                    tcgen05_fence_after();
                    const uint32_t k_s = sb + Cfg::OFF_K + s * Cfg::KV_BYTES;
                    const uint32_t v_s = sb + Cfg::OFF_V + s * Cfg::KV_BYTES;
#pragma unroll
                    for (int q = 0; q < NQ; ++q) {
                        if (t > it.t0[q] && t <= it.t1[q]) {
                            // O_q += P_q(t-1) V_(t-1)
                            if (!(ok = w.wait(bars.pfull(q), pv_n[q] & 1u, kDevErrMmaFull))) break;
                            ++pv_n[q];
                            tcgen05_fence_after();
                            const uint32_t p_t = tmem_base + Cfg::T_S + q * 128 + Cfg::P_COL;
#pragma unroll
                            for (int k = 0; k < Cfg::BKV / 16; ++k)
                                mma_f16_ts(tmem_base + Cfg::T_O + q * D, p_t + k * 8,
                                           smem_desc_sw128(v_s + k * 2048, Cfg::CHUNK_BYTES, 1024), Cfg::IDESC_PV,
                                           (t - 1 > it.t0[q] || k > 0) ? 1u : 0u);
                            if (t == it.t1[q]) mma_commit(bars.odone(q));
                        }
                        if (t >= it.t0[q] && t < it.t1[q]) {
                            // S_q(t) = Q_q K_t^T, over P_q(t-1): one thread's products complete in order
                            const uint32_t q_s = sb + Cfg::OFF_Q + (qb * NQ + q) * Cfg::Q_BYTES;
#pragma unroll
                            for (int k = 0; k < D / 16; ++k) {
                                const uint32_t off = (k >> 2) * Cfg::CHUNK_BYTES + (k & 3) * 32;
                                mma_f16_ss(tmem_base + Cfg::T_S + q * 128, smem_desc_sw128(q_s + off, 16, 1024),
                                           smem_desc_sw128(k_s + off, 16, 1024), Cfg::IDESC_S, k > 0 ? 1u : 0u);
                            }
                            mma_commit(bars.sfull(q));
                        }
                    }
                    if (!ok) break;
                    if (t == t_end - 1) mma_commit(bars.qfree(qb));   // the item's last Q K^T products are issued
                    mma_commit(bars.empty(s));
                }
            }
            mma_commit(bars.drain());
            w.drain(bars.drain(), 0);
        }
        __syncwarp();
    };

    auto softmax = [&](auto run) {
        constexpr bool SECOND = decltype(run)::value;
        const FwdBars bars{sb + (SECOND ? Cfg::OFF_BAR_AGAIN : Cfg::OFF_BAR)};
        // ------------------------------------------------------------ softmax + output (warps 4-11)
        const int q = (warp - 4) >> 2;
        const int quad = warp & 3;
        const int r = quad * 32 + lane;
        const uint32_t lane_base = tmem_base + ((uint32_t)(quad * 32) << 16);
        const uint32_t s_col = lane_base + Cfg::T_S + q * 128;
        const uint32_t o_col = lane_base + Cfg::T_O + q * D;
        const ScoreArgs& sc = p.score;
        const ScoreForm form = score_form<Cfg::MODE>(sc);
        const uint32_t hidden = form.hidden();
        uint32_t n_item = 0, s_n = 0, o_n = 0;
        bool ok = true;
        while (ok) {
            const uint32_t box = n_item & 1u;
            if (!__all_sync(0xffffffffu, w.wait(bars.item_pub(box), (n_item >> 1) & 1u, kDevErrEpilogueFull))) break;
            const Item it = read_item(box);
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.item_read(box));
            ++n_item;
            if (it.b < 0) break;
            const int qi = it.q_base + q * Cfg::BQ + r;
            const int t0 = q == 0 ? it.t0[0] : it.t0[1], t1 = q == 0 ? it.t1[0] : it.t1[1];
            int lo = 0, hi = 0;
            if (qi < mk.Sq && t0 < t1) row_interval(mk, it.b, qi, lo, hi);
            const float slope2 = kHasBias<Cfg::MODE> ? __ldg(sc.slopes + it.h) * kLog2e : 0.0f;
            float m = -INFINITY, l = 0.0f;

            for (int t = t0; t < t1; ++t) {
                // the warp agrees before any .sync.aligned TMEM access
                if (!__all_sync(0xffffffffu, w.wait(bars.sfull(q), s_n & 1u, kDevErrEpilogueFull))) {
                    ok = false;
                    break;
                }
                ++s_n;
                tcgen05_fence_after();
                const int k0 = it.key_tile(t) * Cfg::BKV;
                const bool masked = __any_sync(0xffffffffu, k0 < lo || k0 + Cfg::BKV > hi);
                uint32_t sc0[32], sc1[32], sc2[32], sc3[32];
                tmem_ld_32x32b_x32(s_col + 0, sc0);
                tmem_ld_32x32b_x32(s_col + 32, sc1);
                tmem_ld_32x32b_x32(s_col + 64, sc2);
                tmem_ld_32x32b_x32(s_col + 96, sc3);
                tmem_ld_wait(sc0);
                reg_tie(sc1);
                reg_tie(sc2);
                reg_tie(sc3);
                const float base = (float)(qi + mk.offset - k0);
                score_row<Cfg::MODE, true>(sc0, sc1, sc2, sc3, sc, slope2, base);
                if (masked) {
                    // of a boundary tile's four chunks few hold the boundary, and the warp's rows share it
                    auto hide = [&](uint32_t (&rr)[32], int c) {
                        const uint32_t vis = between(lo - k0 - c * 32, hi - k0 - c * 32);
                        if (__all_sync(0xffffffffu, vis == 0xffffffffu)) return;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!(vis >> i & 1u)) rr[i] = hidden;
                    };
                    hide(sc0, 0);
                    hide(sc1, 1);
                    hide(sc2, 2);
                    hide(sc3, 3);
                }
                float mt = form.ascending ? row_max(sc0, sc1, sc2, sc3) : row_min(sc0, sc1, sc2, sc3);
                mt *= form.mul;
                // lazy move of the exponent base: only by more than 2^RESCALE_LOG2 (always from -inf)
                float factor = 1.0f;
                const bool bump = mt > m + Cfg::RESCALE_LOG2;
                if (bump) {
                    factor = (m == -INFINITY) ? 0.0f : ex2_approx(m - mt);
                    m = mt;
                }
                l *= factor;
                const float neg_m = (m == -INFINITY) ? 0.0f : -m, mul = form.mul;
                float ls0 = 0.0f, ls1 = 0.0f;
                auto chunk_p = [&](const uint32_t (&rr)[32], int c) {
                    uint32_t packed[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float x0, x1;
                        ffma2(x0, x1, __uint_as_float(rr[2 * i]), __uint_as_float(rr[2 * i + 1]), mul, mul, neg_m, neg_m);
                        const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                        fadd2(ls0, ls1, p0, p1);
                        packed[i] = Elem<T>::pack(p0, p1);
                    }
                    tmem_st_32x32b_x16(s_col + Cfg::P_COL + c * 16, packed);
                };
                __syncwarp();                    // whole warps at the TMEM accesses
                chunk_p(sc0, 0);
                chunk_p(sc1, 1);
                chunk_p(sc2, 2);
                chunk_p(sc3, 3);
                if (t > t0 && __any_sync(0xffffffffu, bump)) {
                    // O_q (this warp's rows) *= factor: PV_q(t-1) completed before S_q(t) did, and
                    // PV_q(t) waits for the arrival below; done after the exponentials, when the
                    // scores are dead
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t rr[32];
                        tmem_ld_32x32b_x32(o_col + c * 32, rr);
                        tmem_ld_wait(rr);
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            float y0, y1;
                            fmul2(y0, y1, __uint_as_float(rr[i]), __uint_as_float(rr[i + 1]), factor, factor);
                            rr[i] = __float_as_uint(y0);
                            rr[i + 1] = __float_as_uint(y1);
                        }
                        tmem_st_32x32b_x32(o_col + c * 32, rr);
                    }
                }
                tmem_st_wait();
                tcgen05_fence_before();
                mbar_arrive(bars.pfull(q));           // P_q(t) (and a rescaled O_q) ready for the MMA
                l += ls0 + ls1;
            }
            // output: O_q / l, and the log-sum-exp.  The next item's first PV_q, which overwrites
            // O_q, waits for this group's next P, issued only after these loads.
            if (ok && t0 < t1) {
                ok = __all_sync(0xffffffffu, w.wait(bars.odone(q), o_n & 1u, kDevErrEpilogueFull));
                ++o_n;
                tcgen05_fence_after();
            }
            if (!ok) break;
            if (p.splits > 1) {
                const bool bad = store_part<D>(p, part_index(p, it.b, it.h, it.split, qi), t0 < t1, qi < mk.Sq, o_col, m, l);
                if (SECOND || __any_sync(0xffffffffu, bad && qi < mk.Sq && l < INFINITY))
                    after_item<Cfg, SECOND>(p, n_item, it.b, it.h, it.q_base, it.split);
                continue;
            }
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            bool bad = false;                    // an element of O is infinite or NaN
            T* dst = static_cast<T*>(p.O.data) + it.b * p.O.batch + it.h * p.O.head + (long long)qi * p.O.row;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {   // one copy of the code: it runs cold, once an item
                uint32_t rr[32];
                __syncwarp();
                if (t0 < t1) {
                    tmem_ld_32x32b_x32(o_col + c * 32, rr);
                    tmem_ld_wait(rr);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) rr[i] = 0u;
                }
                if (lo >= hi) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) rr[i] = 0u;     // 0 V of a row without keys
                }
                if (qi < mk.Sq) {
                    uint32_t v[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float a = __uint_as_float(rr[2 * i]), b = __uint_as_float(rr[2 * i + 1]);
                        bad |= !(fabsf(a) < INFINITY) | !(fabsf(b) < INFINITY);
                        v[i] = Elem<T>::pack(a * inv, b * inv);
                    }
                    store_64_bytes(dst + c * 32, v);
                }
            }
            if (p.lse && qi < mk.Sq)
                p.lse[((long long)it.b * mk.Hq + it.h) * mk.Sq + qi] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
            tcgen05_fence_before();
            // a row whose sum is not finite owes it to its scores alone
            if (SECOND || __any_sync(0xffffffffu, bad && qi < mk.Sq && l < INFINITY))
                after_item<Cfg, SECOND>(p, n_item, it.b, it.h, it.q_base, it.split);
        }
    };

    // Roles run once, and again if the list is not empty.  At the barrier between, all of the first run is written, its
    // copies have landed and its products are done.  The order of the code below decides how far the second
    // run's copy lies from the first's loops: 8192 tokens in documents, capped, 174.5 us; each role's two runs side by
    // side, the copying and issuing warps first, 178.
    auto first_run = [&](auto role) {
        role(std::false_type{});
        tcgen05_fence_before();
        named_bar_sync(0, Cfg::NUM_THREADS);
        return again_words[0] != 0u && *abort_flag == 0u;
    };
    auto second_run = [&](auto role) {
        if (threadIdx.x == 0) FwdBars{sb + Cfg::OFF_BAR_AGAIN}.init(Cfg::SM_THREADS / 32);
        named_bar_sync(0, Cfg::NUM_THREADS);
        role(std::true_type{});
        tcgen05_fence_before();
        named_bar_sync(0, Cfg::NUM_THREADS);
    };
    if (warp >= 4) {
        reg_inc<Cfg::SOFTMAX_REGS>();
        if (first_run(softmax)) second_run(softmax);
    } else {
        reg_dec<Cfg::CONTROL_REGS>();
        bool more;
        if (warp == 0)
            more = first_run(produce);
        else if (warp == 1)
            more = first_run(issue);
        else
            more = first_run([](auto) {});
        if (more) {
            if (warp == 0)
                second_run(produce);
            else if (warp == 1)
                second_run(issue);
            else
                second_run([](auto) {});
        }
    }
    if (warp == 1) {
        __syncwarp();
        tcgen05_fence_after();
        tmem_dealloc(tmem_base, Cfg::TMEM_COLS);
    }
}

template <class Cfg>
cudaError_t launch_masked_cfg(const MaskedFwdMaps& tm, const MaskedFwdParams& p, cudaStream_t stream) {
    static std::atomic<uint64_t> attr_done{0};
    cudaError_t e = allow_smem(gsr_masked_fwd_kernel<Cfg>, Cfg::SMEM_BYTES, attr_done);
    if (e != cudaSuccess) return e;
    gsr_masked_fwd_kernel<Cfg><<<(unsigned)p.num_items, Cfg::NUM_THREADS, Cfg::SMEM_BYTES, stream>>>(tm.q, tm.k, tm.v, p);
    if ((e = cudaGetLastError()) != cudaSuccess || p.splits == 1) return e;
    const long long rows = (long long)p.mask.B * p.mask.Hq * p.mask.Sq;
    return launch_early(gsr_masked_fwd_join_kernel<typename Cfg::T, Cfg::D>, (unsigned)((rows + 7) / 8), 256, 0, stream, p);
}

template <class T, int D>
cudaError_t launch_masked_type(const MaskedFwdMaps& tm, const MaskedFwdParams& p, cudaStream_t stream) {
    if (p.mask.Skv == 0) {
        const long long rows = (long long)p.mask.B * p.mask.Hq * p.mask.Sq;
        gsr_masked_empty_kernel<T, D><<<(unsigned)((rows + 7) / 8), 256, 0, stream>>>(p);
        return cudaGetLastError();
    }
    switch (score_mode(p.score)) {
        case kScorePlain: return launch_masked_cfg<MaskedFwdCfg<T, D, kScorePlain>>(tm, p, stream);
        case kScoreBias: return launch_masked_cfg<MaskedFwdCfg<T, D, kScoreBias>>(tm, p, stream);
        case kScoreCap: return launch_masked_cfg<MaskedFwdCfg<T, D, kScoreCap>>(tm, p, stream);
        default: return launch_masked_cfg<MaskedFwdCfg<T, D, kScoreCapBias>>(tm, p, stream);
    }
}

}  // namespace gsr
