// attention_tree.cuh - attention of drafted tokens over a paged key/value cache.  Instantiated per
// element type and head_dim.
//
// Request b has kv_lens[b] cached tokens; the last T_b of them are its drafted tokens, the nodes of
// a tree (q_starts gives the packed query rows, parents each node's parent).  A node sees the
// tokens before the tree, its ancestors and itself; T_b = 1 is ordinary decoding.
//
// Bound by the read of K and V: the query heads of a group and all nodes of a request share them,
// so they are the rows of one 128-row query tile (row = node x group + head of the group), and a
// key tile read once serves all of them.  A 128 x 128 x D product pair takes 1/3 of the time in
// which an SM gets its share of HBM bandwidth for the tile, even with one row of the 128 in use.
// Requests of more than 128 rows run two query tiles per pass (NQ = 2).
//
// Two softmax groups of four warps work on alternate products.  With two query tiles each has its
// own; with one they take turns over the key tiles, each with its own maximum, sum and accumulator
// (even and odd key tiles are two parts of one softmax), and add up at the end: one group alone
// took 2500 cycles a key tile at D = 64, where HBM brings one in 1500.
//
//  * Work is split evenly whatever the lengths: all (request, key/value head, pair of query tiles)
//    items' key tiles are laid end to end, and CTA c of G takes the range [U c / G, U (c+1) / G).
//    Every CTA finds its range from kv_lens and q_starts by one sum over the requests, so the host
//    needs no lengths and a captured launch follows them.
//  * An item that one CTA covers whole is written at once.  Otherwise each of its CTAs leaves its
//    part (sum, maximum, O in fp32) in the workspace, at most two a CTA (its range's first and last
//    item), and a second launch joins them in the order of the CTAs.
//  * Pages arrive by TMA, one box per page (or piece of one), a ring of key and value tiles ahead of
//    the tensor core; lane i of the producer warp looks up and copies piece i of the tile.  A box
//    costs the copy unit about 85 cycles whatever it holds, so at head_dim 128 it takes both 64-column
//    chunks of its rows: a tile lies in shared memory as groups of 8 rows, each group's chunks side by
//    side (one box a chunk: pages of 8 rows 321 us where HBM needs 170, of 16 rows 214).
//  * Rows of the last tile behind kv_lens, and pieces whose page is not in the pool, are masked, and
//    their V rows set to zero in shared memory before the product (0 times what a page holds there
//    may be NaN).  Of the tiles that hold nodes of a tree, where nodes do not see their siblings, the elements of V
//    that are not finite are ("Infinities and NaN behind a mask" in attention_common.cuh).
#pragma once

#include "attention_common.cuh"
#include "ptx_attention.cuh"

namespace gsr {

// ---------------------------------------------------------------------------
// Requests
// ---------------------------------------------------------------------------
struct TreeRequest {
    int start;      // first query row
    int count;      // drafted tokens
    int nodes;      // of them computed: count, at most max_nodes
    int kv;         // cached tokens the table can hold
    int ctx;        // tokens before the tree (may be negative where kv_lens is below count)
    int q_pairs;    // pairs (NQ = 2) or single (NQ = 1) query tiles
    int key_tiles;
    __device__ __forceinline__ long long units(int heads) const { return (long long)heads * q_pairs * key_tiles; }
};

__device__ __forceinline__ TreeRequest tree_request(const TreeParams& p, int b) {
    TreeRequest r;
    r.start = max(__ldg(p.q_starts + b), 0);
    const int end = min(__ldg(p.q_starts + b + 1), p.total_q);
    const int len = max(__ldg(p.kv_lens + b), 0);
    r.count = max(end - r.start, 0);
    r.nodes = min(r.count, p.max_nodes);
    r.kv = min(len, p.table_width * p.page);
    r.ctx = len - r.count;
    const int per_pass = p.tile_nodes * p.nq;
    r.q_pairs = (r.nodes + per_pass - 1) / per_pass;
    r.key_tiles = max((r.kv + p.tile_keys - 1) / p.tile_keys, 1);
    return r;
}

// Bit u: node u is node t or one of its ancestors.  A parent that is no earlier node ends the walk.
__device__ __forceinline__ uint64_t ancestors(const int* parents, int start, int t) {
    if (!parents) return t >= 63 ? ~0ull : (2ull << t) - 1;
    uint64_t bits = 1ull << t;
    for (int u = t;;) {
        const int up = __ldg(parents + start + u);
        if (up < 0 || up >= u) return bits;
        bits |= 1ull << up;
        u = up;
    }
}

// The depth of node t's ancestor (or of t itself) u: its own ancestors are those of t before it.
__device__ __forceinline__ int depth_of(uint64_t see, int u) { return __popcll(see & ((1ull << u) - 1)); }

// ---------------------------------------------------------------------------
// Configuration
// ---------------------------------------------------------------------------
template <class T_, int D_, int MODE_, int NQ_>
struct TreeCfg {
    using T = T_;
    static constexpr int D = D_, MODE = MODE_, NQ = NQ_;
    static constexpr int DCH = D / 64;
    static constexpr int CHUNK_BYTES = 128 * 128;     // a query tile's 64 columns
    static constexpr int TILE_BYTES = 128 * D * 2;
    static constexpr int GROUP_BYTES = 8 * D * 2;     // 8 rows of a key or value tile
    static constexpr int NB = D == 128 ? (NQ == 1 ? 6 : 5) : 12;   // ring of K and V tiles
    static constexpr int SM_THREADS = 256;            // two softmax groups of four warps
    static constexpr int NUM_THREADS = 128 + SM_THREADS;
    // 384 threads start with 168 registers each; the copying and issuing warps' group gives some to
    // the softmax groups, whose threads hold a row of 128 scores: 72 + 2 x 216 = 3 x 168
    static constexpr int CONTROL_REGS = 72, SOFTMAX_REGS = 216;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_RING = OFF_Q + NQ * TILE_BYTES;
    static constexpr int OFF_BAR = OFF_RING + NB * TILE_BYTES;
    static constexpr int NUM_BARS = 2 * NB + 18;
    static constexpr int OFF_VALID = OFF_BAR + NUM_BARS * 8;       // per ring entry: which pieces of the tile exist
    static constexpr int OFF_ITEM = OFF_VALID + NB * 4;            // 2 x 12 ints
    static constexpr int OFF_SCAN = (OFF_ITEM + 96 + 7) / 8 * 8;   // 16 partial sums, then the CTA's first unit
    static constexpr int OFF_ML = OFF_SCAN + 16 * 8 + 16;          // 2 groups x 128 rows of (m, l)
    static constexpr int OFF_CLEANED = OFF_ML + 2 * 128 * 8;       // 4 words
    static constexpr int OFF_MISC = OFF_CLEANED + 16;
    static constexpr int SMEM_BYTES = OFF_MISC + 16;
    static constexpr uint32_t T_S = 0, T_O = 256, P_COL = 64;
    static constexpr uint32_t IDESC_S = idesc_16_f32(Elem<T>::bf16, 128, 128, false, false);
    static constexpr uint32_t IDESC_PV = idesc_16_f32(Elem<T>::bf16, 128, D, false, true);
    static constexpr float RESCALE_LOG2 = 8.0f;
    static_assert(SMEM_BYTES <= 232448, "shared memory");
};

// Part of an item in the workspace: for each row of its query tiles O (fp32, not normalised) and
// the exponent base m and sum l.
__device__ __forceinline__ float* part_o(const TreeParams& p, long long slot, int row, int D) {
    return p.parts + (slot * p.part_rows + row) * D;
}
__device__ __forceinline__ float2* part_ml(const TreeParams& p, long long slot, int row) {
    return p.parts_ml + slot * p.part_rows + row;
}

// A warp's quarter of a V tile without what is not finite; where there is something, *flag = n first.  With two query
// tiles each softmax group does it before its own product: one that finds the other's zeros finds its flag too.
template <class T, int D>
__device__ __noinline__ void clean_quarter(uint8_t* at, volatile uint32_t* flag, uint32_t n, int lane) {
    __syncwarp();                                        // its lanes may have zeroed rows without a token
    if (pieces_not_finite<T>(at, 4 * D, lane)) {
        *flag = n;
        __threadfence_block();
        __syncwarp();
        zero_not_finite<T>(at, 4 * D, lane);
    }
    fence_proxy_async_smem();                            // the other group's zeros, too, come before this one's product
}

// A warp's rows of an item are written (from column block c0 of 32 on, up to c1), and tiles with nodes were cleaned: what
// their V means to the nodes that see them.  `tile_node` is the first node of the warp's query tile, `part_row`
// that tile's first row in slot `slot` (below 0: the item is whole); key tiles [t0, t1) are the item's.
template <class T, int D>
__device__ __noinline__ void spread_nodes(const TreeParams& p, int b, int hk, int tile_node, int t0, int t1, int slot, int part_row, int c0,
                                          int c1) {
    const int lane = threadIdx.x & 31, rq = (threadIdx.x >> 5 & 3) * 32 + lane;
    const TreeRequest r = tree_request(p, b);
    const int node_in = rq / p.group, node = tile_node + node_in, h = hk * p.group + rq - node_in * p.group;
    const bool real = node_in < p.tile_nodes && node < r.nodes;
    const uint64_t see = real ? ancestors(p.parents, r.start, node) : 0ull;
    Marks<D> marks;
    // from the first cleaned tile on; what is before the tree every node sees
    for (int j0 = max(r.ctx, 0) / p.tile_keys * p.tile_keys, end = min(r.kv, r.ctx + 64); j0 < end; j0 += 4) {
        uint16_t x[4][D / 32];
        bool sees[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int j = min(j0 + k, end - 1), t = j / p.tile_keys, page = __ldg(p.table + (long long)b * p.table_width + j / p.page);
            const bool there = t >= t0 && t < t1 && page >= 0 && page < p.num_pages;
            sees[k] = there && real && (j < r.ctx || (see >> (j - r.ctx) & 1));
            const unsigned short* v = static_cast<const unsigned short*>(p.V.data) + (there ? page : 0) * p.V.batch + (j % p.page) * p.V.row +
                                      hk * p.V.head;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) x[k][c] = there ? __ldg(v + c * 32 + lane) : (unsigned short)0;
        }
        marks.template take<T, false, 4>(x, sees);
    }
    if (real && slot >= 0) marks.template apply<T>(part_o(p, slot, part_row + rq, D), c0, c1);
    if (real && slot < 0)
        marks.template apply<T>(static_cast<uint16_t*>(p.O) + (long long)(r.start + node) * p.o_row + h * p.o_head, c0, c1);
    __syncwarp();
}

// Of a grid's CTAs as many as there are units take part, so each has one at least.  CTA c's first
// unit of U, and the CTA that holds unit u.
__device__ __forceinline__ int busy_ctas(long long U, int grid) { return (int)min((long long)grid, U); }
__device__ __forceinline__ long long first_unit(long long U, int c, int G) { return U * c / G; }
__device__ __forceinline__ int cta_of(long long U, long long u, int G) { return (int)(((u + 1) * G - 1) / U); }

// ---------------------------------------------------------------------------
// The parts
// ---------------------------------------------------------------------------
template <class Cfg>
__global__ void __launch_bounds__(Cfg::NUM_THREADS, 1)
    gsr_tree_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ TreeParams p) {
    using T = typename Cfg::T;
    constexpr int D = Cfg::D, NQ = Cfg::NQ, NB = Cfg::NB, DCH = Cfg::DCH;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023u) {
        if (threadIdx.x == 0) atomicCAS(p.err, 0, kDevErrKernelTree | kDevErrLayout);
        return;
    }
    grid_launch_next();                                          // the joining CTAs, as SMs fall free
    const uint32_t sb = smem_u32(smem);
    auto bar = [&](int i) { return sb + Cfg::OFF_BAR + 8u * i; };
    auto full = [&](int s) { return bar(s); };
    auto empty = [&](int s) { return bar(NB + s); };
    auto sfull = [&](int i) { return bar(2 * NB + i); };        // per S region
    auto pfull = [&](int i) { return bar(2 * NB + 2 + i); };
    // per softmax group and parity of the item: a group without a key tile of its own (an item of one) holds
    // nothing up, and the next item's products may be done before it looks
    auto odone = [&](int q, uint32_t item) { return bar(2 * NB + 4 + 2 * q + (int)(item & 1u)); };
    auto item_pub = [&](int i) { return bar(2 * NB + 8 + i); };
    auto item_read = [&](int i) { return bar(2 * NB + 10 + i); };
    const uint32_t q_full = bar(2 * NB + 12), q_free = bar(2 * NB + 13), drain = bar(2 * NB + 14), ml_full = bar(2 * NB + 15),
                   ml_free = bar(2 * NB + 16);
    // The accumulators of an item have been read.  With one query tile both groups read both of them, so that the
    // next item's first product, which overwrites accumulator 0, has to wait for the warps of group 1 too: the P it
    // takes comes from group 0 alone.  Turns over once an item, and the issuing lane looks once an item.
    const uint32_t o_read = bar(2 * NB + 17);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::OFF_MISC);
    volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + Cfg::OFF_MISC + 4);
    volatile int* item_box = reinterpret_cast<volatile int*>(smem + Cfg::OFF_ITEM);
    volatile uint32_t* valid_box = reinterpret_cast<volatile uint32_t*>(smem + Cfg::OFF_VALID);
    // cleaned[n & 3] == n: a tile of item n was cleaned.  (Item n + 4 is published once every warp is past n.)
    volatile uint32_t* cleaned = reinterpret_cast<volatile uint32_t*>(smem + Cfg::OFF_CLEANED);
    long long* scan = reinterpret_cast<long long*>(smem + Cfg::OFF_SCAN);
    long long* first_box = scan + 16;                            // request, unit in it
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // ---- this CTA's range of units
    const int per = (p.B + Cfg::NUM_THREADS - 1) / Cfg::NUM_THREADS;
    const int b0 = min((int)threadIdx.x * per, p.B), b1 = min(b0 + per, p.B);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += tree_request(p, b).units(p.Hkv);
    long long upto = mine;                                       // inclusive sum
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) scan[warp] = upto;
    if (threadIdx.x == 0) {
        for (int s = 0; s < NB; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(sfull(s), 1);
            mbar_init(pfull(s), 128);
            mbar_init(odone(s, 0), 1);
            mbar_init(odone(s, 1), 1);
            mbar_init(item_pub(s), 1);
            mbar_init(item_read(s), 1 + Cfg::SM_THREADS / 32);
        }
        mbar_init(q_full, 1);
        mbar_init(q_free, 1);
        mbar_init(ml_full, Cfg::SM_THREADS / 32);
        mbar_init(ml_free, Cfg::SM_THREADS / 32);
        mbar_init(drain, 1);
        mbar_init(o_read, Cfg::SM_THREADS / 32);
        for (int i = 0; i < 4; ++i) cleaned[i] = 0u;
        *abort_flag = 0u;
        fence_mbarrier_init();
    }
    __syncthreads();
    long long U = 0;
#pragma unroll
    for (int i = 0; i < Cfg::NUM_THREADS / 32; ++i) {
        if (i < warp) upto += scan[i];
        U += scan[i];
    }
    const int G = busy_ctas(U, gridDim.x);
    const long long u_begin = blockIdx.x < G ? first_unit(U, blockIdx.x, G) : U;
    const long long u_end = blockIdx.x < G ? first_unit(U, blockIdx.x + 1, G) : U;
    long long before = upto - mine;
    for (int b = b0; b < b1; ++b) {
        const long long n = tree_request(p, b).units(p.Hkv);
        if (blockIdx.x == 0) p.unit_starts[b] = before;          // for the joining launch
        if (before <= u_begin && u_begin < before + n) {
            first_box[0] = b;
            first_box[1] = u_begin - before;
        }
        before += n;
    }
    if (blockIdx.x == 0 && threadIdx.x == Cfg::NUM_THREADS - 1) p.unit_starts[p.B] = U;
    if (u_begin >= u_end) return;                                // nothing for this CTA (the same for all its threads)

    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish_alloc_permit();
    }
    // rows behind the tile's last piece are never copied: zero for good
    for (int s = 0; s < NB; ++s)
        for (int i = p.tile_keys * D / 8 + threadIdx.x; i < 128 * D / 8; i += Cfg::NUM_THREADS)
            reinterpret_cast<uint4*>(smem + Cfg::OFF_RING + s * Cfg::TILE_BYTES)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    tcgen05_fence_before();
    __syncthreads();
    tcgen05_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const Waiter w{p.err, p.timeout_ns, abort_flag, kDevErrKernelTree};

    // What the producer publishes; b < 0: no more items.  Key tiles [t0, t1) of the item's `tiles`,
    // query tiles from node n0 on; slot < 0: the item is whole.
    struct Item {
        int b, hk, n0, t0, t1, tiles, start, nodes, kv, ctx, slot, q_tiles;
    };
    auto read_item = [&](int box) {
        volatile int* v = item_box + 12 * box;
        return Item{v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7], v[8], v[9], v[10], v[11]};
    };

    if (warp < 4) {
        reg_dec<Cfg::CONTROL_REGS>();
        if (warp == 0) {
            // ------------------------------------------------------------ items + TMA producer
            const uint64_t pol = l2_policy_evict_normal();
            const int pieces = p.tile_keys / p.piece, per_page = p.page / p.piece;
            uint32_t n_pub = 0, n = 0;                       // items published, tiles
            uint32_t armed = 0, parity = 0;
            bool drop = (p.test_flags & kTestDropFirstLoad) && blockIdx.x == 0;
            bool ok = true;
            int b = (int)first_box[0];
            long long off = first_box[1];
            TreeRequest r = tree_request(p, b);
            for (long long u = u_begin;;) {
                Item it{-1, 0, 0, 0, 0, 0, 0, 0, 0, 0, -1, 0};
                while (u < u_end && b < p.B && off >= r.units(p.Hkv)) {      // the range goes on in a later request
                    off = 0;
                    if (++b < p.B) r = tree_request(p, b);
                }
                if (u < u_end && b < p.B) {
                    const int index = (int)(off / r.key_tiles);
                    it.b = b;
                    it.hk = index / r.q_pairs;
                    it.n0 = (index - it.hk * r.q_pairs) * p.tile_nodes * NQ;
                    it.t0 = (int)(off - (long long)index * r.key_tiles);
                    it.t1 = (int)min((long long)r.key_tiles, it.t0 + (u_end - u));
                    it.tiles = r.key_tiles;
                    it.start = r.start;
                    it.nodes = r.nodes;
                    it.kv = r.kv;
                    it.ctx = r.ctx;
                    it.q_tiles = NQ == 1 || r.nodes - it.n0 <= p.tile_nodes ? 1 : 2;
                    if (it.t0 > 0 || it.t1 < it.tiles) it.slot = 2 * blockIdx.x + (u > u_begin ? 1 : 0);
                }
                const uint32_t box = n_pub & 1u;
                ok = lane != 0 || w.wait(item_read(box), ((n_pub >> 1) & 1u) ^ 1u, kDevErrProducerEmpty);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                if (lane == 0) {
                    volatile int* v = item_box + 12 * box;
                    v[0] = it.b;
                    v[1] = it.hk;
                    v[2] = it.n0;
                    v[3] = it.t0;
                    v[4] = it.t1;
                    v[5] = it.tiles;
                    v[6] = it.start;
                    v[7] = it.nodes;
                    v[8] = it.kv;
                    v[9] = it.ctx;
                    v[10] = it.slot;
                    v[11] = it.q_tiles;
                    mbar_arrive(item_pub(box));
                }
                ++n_pub;
                if (it.b < 0) break;
                // this lane's piece of the next tile: its page, and whether it exists
                auto look_up = [&](int t, int& page, int& row) {
                    const int at = t * pieces + lane;        // piece of the request
                    page = -1;
                    if (lane < pieces && at * p.piece < it.kv) page = __ldg(p.table + (long long)it.b * p.table_width + at / per_page);
                    if (page >= p.num_pages) page = -1;
                    row = at % per_page * p.piece;
                };
                int page, row, next_page, next_row;
                look_up(it.t0, page, row);
                if (lane == 0) {
                    ok = n_pub == 1 || w.wait(q_free, n_pub & 1u, kDevErrProducerEmpty);   // the previous item's
                    if (ok && !drop) {
                        mbar_arrive_expect_tx(q_full, it.q_tiles * p.tile_nodes * p.group * 128 * DCH);
                        for (int q = 0; q < it.q_tiles; ++q)
#pragma unroll
                            for (int c = 0; c < DCH; ++c)
                                tma_load_4d(sb + Cfg::OFF_Q + q * Cfg::TILE_BYTES + c * Cfg::CHUNK_BYTES, &tmQ, q_full, c * 64, 0,
                                            it.hk, it.start + it.n0 + q * p.tile_nodes, pol);
                        armed |= 1u << NB;
                        parity = (parity & ~(1u << NB)) | ((n_pub - 1) & 1u) << NB;
                    }
                    drop = false;                            // test hook: the first Q is never loaded
                }
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                for (int t = it.t0; t < it.t1; ++t, ++n) {
                    look_up(t + 1 < it.t1 ? t + 1 : t, next_page, next_row);
                    const uint32_t exists = __ballot_sync(0xffffffffu, page >= 0);
                    const uint32_t bytes = __popc(exists) * p.piece * 128 * DCH;
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        const uint32_t e = 2 * n + kv;
                        const int s = (int)(e % NB);
                        if (lane == 0) {
                            ok = w.wait(empty(s), ((e / NB) & 1u) ^ 1u, kDevErrProducerEmpty);
                            if (ok) {
                                valid_box[s] = exists;
                                mbar_arrive_expect_tx(full(s), bytes);
                            }
                        }
                        if (!(ok = __all_sync(0xffffffffu, ok))) break;
                        armed |= 1u << s;
                        parity = (parity & ~(1u << s)) | ((e / NB) & 1u) << s;
                        if (page >= 0) {
                            const CacheAxes& ax = kv ? p.v_axes : p.k_axes;
                            const int outer = ax.by_head ? it.hk : page;      // what the groups of 8 rows are counted in
                            tma_load_5d(sb + Cfg::OFF_RING + s * Cfg::TILE_BYTES + lane * (p.piece / 8) * Cfg::GROUP_BYTES,
                                        kv ? &tmV : &tmK, full(s), 0, 0, 0, outer * ax.step + row / 8,
                                        ax.by_head ? page : it.hk, pol);
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                    page = next_page;
                    row = next_row;
                }
                if (!ok) break;
                u += it.t1 - it.t0;
                off += it.t1 - it.t0;
            }
            if (lane == 0) {   // every copy under way must land before the CTA may exit
                for (int s = 0; s < NB; ++s)
                    if (armed & (1u << s)) w.drain(full(s), (parity >> s) & 1u);
                if (armed & (1u << NB)) w.drain(q_full, (parity >> NB) & 1u);
            }
            __syncwarp();
        } else if (warp == 1) {
            // ------------------------------------------------------------ MMA issuer
            if (lane == 0) {
                uint32_t n_item = 0, n = 0;
                uint32_t p_n[2] = {0u, 0u};                  // pfull phases waited for, per S region
                bool ok = true;
                auto wait_full = [&](uint32_t e) { return w.wait(full((int)(e % NB)), (e / NB) & 1u, kDevErrMmaFull); };
                auto tile = [&](uint32_t e) { return sb + Cfg::OFF_RING + (e % NB) * Cfg::TILE_BYTES; };
                auto issue_s = [&](int q, int region, uint32_t m) {
                    const uint32_t q_s = sb + Cfg::OFF_Q + q * Cfg::TILE_BYTES, k_s = tile(2 * m);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t o = (k >> 2) * Cfg::CHUNK_BYTES + (k & 3) * 32;
                        mma_f16_ss(tmem_base + Cfg::T_S + region * 128, smem_desc_sw128(q_s + o, 16, 1024),
                                   smem_desc_sw128(k_s + (k >> 2) * 1024 + (k & 3) * 32, 16, Cfg::GROUP_BYTES), Cfg::IDESC_S,
                                   k > 0 ? 1u : 0u);
                    }
                    mma_commit(sfull(region));
                };
                auto issue_pv = [&](int q, int region, uint32_t m, bool first) {
                    if (!w.wait(pfull(region), p_n[region] & 1u, kDevErrMmaFull)) return false;
                    ++p_n[region];
                    tcgen05_fence_after();
                    const uint32_t v_s = tile(2 * m + 1), p_t = tmem_base + Cfg::T_S + region * 128 + Cfg::P_COL;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mma_f16_ts(tmem_base + Cfg::T_O + q * D, p_t + k * 8,
                                   smem_desc_sw128(v_s + k * 2 * Cfg::GROUP_BYTES, 1024, Cfg::GROUP_BYTES), Cfg::IDESC_PV,
                                   (!first || k > 0) ? 1u : 0u);
                    return true;
                };
                while (ok) {
                    const uint32_t box = n_item & 1u;
                    if (!w.wait(item_pub(box), (n_item >> 1) & 1u, kDevErrMmaFull)) break;
                    const Item it = read_item(box);
                    mbar_arrive(item_read(box));
                    if (it.b < 0) break;
                    if (!w.wait(q_full, n_item & 1u, kDevErrMmaFull)) break;
                    ++n_item;
                    tcgen05_fence_after();
                    const int steps = it.t1 - it.t0;
                    for (int i = 0; i <= steps && ok; ++i) {
                        // K of step i and V of step i - 1
                        if (i < steps && !(ok = wait_full(2 * (n + i)))) break;
                        tcgen05_fence_after();
                        // the first product of an item overwrites what the last one's rows were read from
                        auto accumulators_read = [&] { return i != 1 || n_item == 1 || w.wait(o_read, n_item & 1u, kDevErrMmaFull); };
                        if (it.q_tiles == 1) {
                            // key tiles in turn: S(i) runs while the other group's softmax does
                            if (i < steps) {
                                issue_s(0, i & 1, n + i);
                                mma_commit(empty((int)(2 * (n + i) % NB)));
                                if (i == steps - 1) mma_commit(q_free);
                            }
                            if (i > 0) {
                                const uint32_t m = n + i - 1;
                                const int g = (i - 1) & 1;
                                if (!(ok = wait_full(2 * m + 1) && accumulators_read() && issue_pv(g, g, m, i <= 2))) break;
                                mma_commit(empty((int)((2 * m + 1) % NB)));
                                if (i == steps) {
                                    mma_commit(odone(0, n_item - 1));
                                    mma_commit(odone(1, n_item - 1));
                                }
                            }
                        } else {
                            // a region per query tile: the tiles alternate on the tensor core
                            if (i > 0 && !(ok = wait_full(2 * (n + i) - 1) && accumulators_read())) break;
                            tcgen05_fence_after();
                            for (int q = 0; q < 2 && ok; ++q) {
                                if (i > 0) {
                                    if (!(ok = issue_pv(q, q, n + i - 1, i == 1))) break;
                                    if (i == steps) mma_commit(odone(q, n_item - 1));
                                }
                                if (i < steps) issue_s(q, q, n + i);
                            }
                            if (!ok) break;
                            if (i < steps) mma_commit(empty((int)(2 * (n + i) % NB)));
                            if (i == steps - 1) mma_commit(q_free);
                            if (i > 0) mma_commit(empty((int)((2 * (n + i) - 1) % NB)));
                        }
                    }
                    n += steps;
                }
                mma_commit(drain);
                w.drain(drain, 0);
            }
            __syncwarp();
        }
    } else {
        reg_inc<Cfg::SOFTMAX_REGS>();
        // ------------------------------------------------------------ softmax + output
        const int q = (warp - 4) >> 2;
        const int quad = warp & 3;
        const int rq = quad * 32 + lane;                 // row of the query tile == TMEM lane
        const uint32_t lane_base = tmem_base + ((uint32_t)(quad * 32) << 16);
        const uint32_t o_col = lane_base + Cfg::T_O + q * D;
        const ScoreArgs& sc = p.score;
        const ScoreForm form = score_form<Cfg::MODE>(sc);
        const uint32_t hidden = form.hidden();
        const int node_in = rq / p.group, hg = rq - node_in * p.group;
        const uint32_t s_col = lane_base + Cfg::T_S + q * 128;
        float2* ml_box = reinterpret_cast<float2*>(smem + Cfg::OFF_ML);
        uint32_t n_item = 0, n_first = 0, s_n = 0, n_ml = 0;     // items, the item's first tile, S phases, exchanges
        bool ok = true;
        while (ok) {
            const uint32_t box = n_item & 1u;
            if (!__all_sync(0xffffffffu, w.wait(item_pub(box), (n_item >> 1) & 1u, kDevErrEpilogueFull))) break;
            const Item it = read_item(box);
            __syncwarp();
            if (lane == 0) mbar_arrive(item_read(box));
            ++n_item;
            if (it.b < 0) break;
            const int steps = it.t1 - it.t0;
            const bool turns = it.q_tiles == 1;          // the groups take turns over the key tiles
            const int node = it.n0 + (turns ? 0 : q * p.tile_nodes) + node_in;
            const bool real = node_in < p.tile_nodes && node < it.nodes;
            const bool busy = __any_sync(0xffffffffu, real);     // warps without rows only keep the barriers
            const int h = it.hk * p.group + hg;
            const uint64_t see = real ? ancestors(p.parents, it.start, node) : 0ull;
            const float slope2 = kHasBias<Cfg::MODE> && real ? __ldg(sc.slopes + h) * kLog2e : 0.0f;
            const int pos = it.ctx + __popcll(see) - 1;
            const int seen_by_all = min(it.ctx, it.kv);  // keys before it are visible to every node
            float m = -INFINITY, l = 0.0f;

            const int i_first = turns ? q : 0, i_step = turns ? 2 : 1;
            for (int i = i_first; i < steps; i += i_step) {
                const uint32_t e = 2 * (n_first + i) + 1;        // V's ring entry
                const int k0 = (it.t0 + i) * p.tile_keys;
                // V's entry tells which pieces exist, and stays until this step's P is used
                if (!__all_sync(0xffffffffu, w.wait(sfull(q), s_n & 1u, kDevErrEpilogueFull) &&
                                                 w.wait(full((int)(e % NB)), (e / NB) & 1u, kDevErrEpilogueFull))) {
                    ok = false;
                    break;
                }
                ++s_n;
                const uint32_t exists = valid_box[e % NB];
                tcgen05_fence_after();
                const bool all_exist = exists == (1u << (p.tile_keys / p.piece)) - 1u;
                const bool partial = !all_exist || k0 + p.tile_keys > it.kv;      // some V rows hold no token
                const bool masked = partial || p.tile_keys < 128 || k0 + 128 > seen_by_all;
                bool bump = false;
                float factor = 1.0f;
                if (busy) {
                    uint32_t sc0[32], sc1[32], sc2[32], sc3[32];
                    tmem_ld_32x32b_x32(s_col + 0, sc0);
                    tmem_ld_32x32b_x32(s_col + 32, sc1);
                    tmem_ld_32x32b_x32(s_col + 64, sc2);
                    tmem_ld_32x32b_x32(s_col + 96, sc3);
                    tmem_ld_wait(sc0);
                    reg_tie(sc1);
                    reg_tie(sc2);
                    reg_tie(sc3);
                    const float base = (float)(pos - k0);
                    // the polynomial's second copy of the code costs more here, where items are short and find it
                    // cold, than it saves (16 trees of up to 40 nodes: 121 us with it, 111 without)
                    score_row<Cfg::MODE, false>(sc0, sc1, sc2, sc3, sc, slope2, base);
                    auto hide = [&](uint32_t (&rr)[32], int c) {
                        const int kk = k0 + c * 32;
                        auto below = [&](int limit) {    // keys before `limit`
                            const int k = limit - kk;
                            return k >= 32 ? 0xffffffffu : (k <= 0 ? 0u : (1u << k) - 1u);
                        };
                        uint32_t tree = 0u;              // the tree's keys among these 32
                        const int sh = kk - it.ctx;
                        if (sh >= 0 && sh < 64) tree = (uint32_t)(see >> sh);
                        if (sh < 0 && sh > -32) tree = (uint32_t)(see << -sh);
                        if (kHasBias<Cfg::MODE> && tree) {
                            // a node's distance counts its depth, not its place in the cache
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (tree >> j & 1u) {
                                    const float at = (float)(pos - it.ctx - depth_of(see, sh + j));
                                    rr[j] = __float_as_uint(fmaf(slope2, fabsf(base - (float)(c * 32 + j)) - at, __uint_as_float(rr[j])));
                                }
                        }
                        uint32_t vis = (tree | below(it.ctx)) & below(min(it.kv, k0 + p.tile_keys));
                        if (!all_exist) {
#pragma unroll 1
                            for (int g8 = 0; g8 < 4; ++g8)
                                if (!(exists >> ((c * 32 + g8 * 8) / p.piece) & 1u)) vis &= ~(0xffu << (8 * g8));
                        }
                        if (vis == 0xffffffffu) return;
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (!(vis >> j & 1u)) rr[j] = hidden;
                    };
                    if (masked) {
                        hide(sc0, 0);
                        hide(sc1, 1);
                        hide(sc2, 2);
                        hide(sc3, 3);
                    }
                    const float mt = (form.ascending ? row_max(sc0, sc1, sc2, sc3) : row_min(sc0, sc1, sc2, sc3)) * form.mul;
                    bump = mt > m + Cfg::RESCALE_LOG2;   // always from -inf
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
                        for (int j = 0; j < 16; ++j) {
                            float x0, x1;
                            ffma2(x0, x1, __uint_as_float(rr[2 * j]), __uint_as_float(rr[2 * j + 1]), mul, mul, neg_m, neg_m);
                            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                            fadd2(ls0, ls1, p0, p1);
                            packed[j] = Elem<T>::pack(p0, p1);
                        }
                        tmem_st_32x32b_x16(s_col + Cfg::P_COL + c * 16, packed);
                    };
                    __syncwarp();                        // whole warps at the TMEM accesses
                    chunk_p(sc0, 0);
                    chunk_p(sc1, 1);
                    chunk_p(sc2, 2);
                    chunk_p(sc3, 3);
                    l += ls0 + ls1;
                }
                if (i > i_first && __any_sync(0xffffffffu, bump)) {
                    // O (this warp's rows) *= factor: the group's last PV was issued before this S, and
                    // its next waits for the arrival below
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t rr[32];
                        tmem_ld_32x32b_x32(o_col + c * 32, rr);
                        tmem_ld_wait(rr);
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            float y0, y1;
                            fmul2(y0, y1, __uint_as_float(rr[j]), __uint_as_float(rr[j + 1]), factor, factor);
                            rr[j] = __float_as_uint(y0);
                            rr[j + 1] = __float_as_uint(y1);
                        }
                        tmem_st_32x32b_x32(o_col + c * 32, rr);
                    }
                }
                if (partial) {
                    // V rows without a token: zero (thread = row of the tile)
                    if (rq < p.tile_keys && (k0 + rq >= it.kv || !(exists >> (rq / p.piece) & 1u))) {
#pragma unroll
                        for (int c = 0; c < DCH; ++c)
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                *reinterpret_cast<uint4*>(smem + Cfg::OFF_RING + (e % NB) * Cfg::TILE_BYTES +
                                                          (rq >> 3) * Cfg::GROUP_BYTES + c * 1024 + (rq & 7) * 128 + j * 16) =
                                    make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
                // a tile with nodes, of a request that has several
                if (it.kv - it.ctx > 1 && k0 + p.tile_keys > it.ctx)
                    clean_quarter<T, D>(smem + Cfg::OFF_RING + (e % NB) * Cfg::TILE_BYTES + quad * (Cfg::TILE_BYTES / 4),
                                        cleaned + (n_item & 3u), n_item, lane);
                tmem_st_wait();
                tcgen05_fence_before();
                mbar_arrive(pfull(q));
            }
            if (!ok) break;
            n_first += steps;
            if (turns) {
                // the two groups' maxima and sums, once both have read the last exchange's
                if (!(ok = __all_sync(0xffffffffu, w.wait(ml_free, (n_ml & 1u) ^ 1u, kDevErrEpilogueFull)))) break;
                ml_box[q * 128 + rq] = make_float2(m, l);
                __syncwarp();
                if (lane == 0) mbar_arrive(ml_full);
            }
            if (!(ok = __all_sync(0xffffffffu, w.wait(odone(q, n_item - 1), ((n_item - 1) >> 1) & 1u, kDevErrEpilogueFull)))) break;
            float f0 = 1.0f, f1 = 0.0f;                  // factors of the two accumulators, and whether they hold anything
            bool use0 = true, use1 = false;
            if (turns) {
                if (!(ok = __all_sync(0xffffffffu, w.wait(ml_full, n_ml & 1u, kDevErrEpilogueFull)))) break;
                const float2 a = ml_box[rq], b = ml_box[128 + rq];
                __syncwarp();
                if (lane == 0) mbar_arrive(ml_free);
                ++n_ml;
                m = fmaxf(a.x, b.x);
                f0 = a.x == -INFINITY ? 0.0f : ex2_approx(a.x - m);
                f1 = b.x == -INFINITY ? 0.0f : ex2_approx(b.x - m);
                use0 = a.x != -INFINITY || a.y != a.y;
                use1 = b.x != -INFINITY || b.y != b.y;
                l = a.y * f0 + b.y * f1;                 // a sum of nothing is 0, or NaN
            }
            tcgen05_fence_after();
            // the rows, or this CTA's part of them; of one query tile's rows each group writes half the
            // columns
            const bool was_cleaned = cleaned[n_item & 3u] == n_item;
            const int c_first = turns ? q * (D / 64) : 0, c_end = turns ? c_first + D / 64 : D / 32;
            if (busy) {
                const float inv = it.slot >= 0 ? 1.0f : (l == 0.0f ? 0.0f : 1.0f / l);
                const bool none = l == 0.0f;             // nothing seen here: O holds 0 V
                f0 *= inv;
                f1 *= inv;
                const uint32_t o0 = turns ? lane_base + Cfg::T_O : o_col, o1 = lane_base + Cfg::T_O + D;
                T* row = static_cast<T*>(p.O) + (long long)(it.start + node) * p.o_row + h * p.o_head;
                float* part = it.slot < 0 ? nullptr : part_o(p, it.slot, (turns ? 0 : q * 128) + rq, D);
#pragma unroll 1
                for (int c = c_first; c < c_end; ++c) {
                    uint32_t r0[32], r1[32];
                    __syncwarp();
                    tmem_ld_32x32b_x32(o0 + c * 32, r0);
                    if (turns && steps > 1) tmem_ld_32x32b_x32(o1 + c * 32, r1);
                    tmem_ld_wait(r0);
                    reg_tie(r1);
                    float y[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        y[j] = !use0 || none ? 0.0f : __uint_as_float(r0[j]) * f0;
                        if (turns && steps > 1 && use1 && !none) y[j] = fmaf(__uint_as_float(r1[j]), f1, y[j]);
                    }
                    if (!real) continue;
                    if (it.slot >= 0) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            reinterpret_cast<float4*>(part)[c * 8 + j] = make_float4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
                    } else {
                        uint32_t v[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) v[k] = Elem<T>::pack(y[2 * k], y[2 * k + 1]);
                        store_64_bytes(row + c * 32, v);
                    }
                }
                if (real && it.slot >= 0 && (!turns || q == 0))
                    *part_ml(p, it.slot, (turns ? 0 : q * 128) + rq) = make_float2(m, l);
            }
            tcgen05_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_read);
            if (busy && was_cleaned)
                spread_nodes<T, D>(p, it.b, it.hk, it.n0 + (turns ? 0 : q * p.tile_nodes), it.t0, it.t1, it.slot, turns ? 0 : q * 128, c_first,
                                   c_end);
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
// Their sum
// ---------------------------------------------------------------------------
// WARPS warps per (query row, head) take its item's parts in the order of their CTAs, warp by warp, and
// add up through shared memory.  A row has few parts where there are many rows, and one warp is
// enough (10 000 rows of 2 or 3 parts: 29 us with four warps a row); a few rows of a long context may
// have a part from every CTA.
constexpr int kJoinThreads = 128;
template <class T, int D, int WARPS>
__global__ void __launch_bounds__(kJoinThreads) gsr_tree_join_kernel(const __grid_constant__ TreeParams p, int grid) {
    constexpr int ROWS = kJoinThreads / 32 / WARPS;
    __shared__ float sm[WARPS > 1 ? WARPS : 1][D + 2];
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % WARPS;
    const long long id = (long long)blockIdx.x * ROWS + (threadIdx.x >> 5) / WARPS;
    // Every CTA waits, also those without a row here: this launch then ends after the parts' launch, and
    // whatever follows it on the stream begins after both.
    if (id >= (long long)p.total_q * p.Hq) {
        grid_wait();
        return;
    }
    const int n = (int)(id / p.Hq), h = (int)(id - (long long)n * p.Hq);
    int left = 0, right = p.B;                                   // first request that ends behind row n
    while (left < right) {
        const int mid = (left + right) >> 1;
        if (__ldg(p.q_starts + mid + 1) <= n) left = mid + 1;
        else right = mid;
    }
    const int b = min(left, p.B - 1);
    const TreeRequest r = tree_request(p, b);
    const int t = n - r.start, hk = h / p.group;
    const int per_pass = p.tile_nodes * p.nq, pair = t / per_pass, in_pass = t - pair * per_pass;
    const int row = in_pass / p.tile_nodes * 128 + in_pass % p.tile_nodes * p.group + (h - hk * p.group);
    grid_wait();                                                 // the parts' launch has finished
    if (left >= p.B || t < 0 || t >= r.nodes) return;            // a row of no request, or of a further node
    const long long U = p.unit_starts[p.B];
    const long long s = p.unit_starts[b] + ((long long)hk * r.q_pairs + pair) * r.key_tiles;
    if (U <= 0) return;
    const int G = busy_ctas(U, grid);
    const int c0 = max(cta_of(U, s, G), 0), c1 = min(cta_of(U, s + r.key_tiles - 1, G), G - 1);
    if (c0 >= c1) return;                                        // written whole
    float m = -INFINITY, l = 0.0f, acc[D / 32] = {};
    auto add = [&](float pm, float pl, const float* o) {
        if (pm == -INFINITY) {                                   // no key that the row sees: the sum is 0, or NaN
            l += pl;
            return;
        }
        const float mn = fmaxf(m, pm);
        const float f0 = m == -INFINITY ? 0.0f : ex2_approx(m - mn), f1 = ex2_approx(pm - mn);
        l = l * (m == -INFINITY ? 1.0f : f0) + pl * f1;          // nothing yet: 0, or NaN
#pragma unroll
        for (int e = 0; e < D / 32; ++e) acc[e] = acc[e] * f0 + o[e] * f1;
        m = mn;
    };
    for (int c = c0 + warp; c <= c1; c += WARPS) {
        const long long slot = 2ll * c + (first_unit(U, c, G) < s ? 1 : 0);
        const float2 ml = *part_ml(p, slot, row);
        const float* o = part_o(p, slot, row, D) + lane * (D / 32);
        float x[D / 32];
#pragma unroll
        for (int e = 0; e < D / 32; ++e) x[e] = o[e];
        add(ml.x, ml.y, x);
    }
    if (WARPS > 1) {
#pragma unroll
        for (int e = 0; e < D / 32; ++e) sm[warp][lane * (D / 32) + e] = acc[e];
        if (lane == 0) {
            sm[warp][D] = m;
            sm[warp][D + 1] = l;
        }
        __syncthreads();
        if (warp != 0) return;
#pragma unroll
        for (int i = 1; i < WARPS; ++i) add(sm[i][D], sm[i][D + 1], &sm[i][lane * (D / 32)]);
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) acc[e] *= inv;
    store_row<T, D>(static_cast<T*>(p.O) + (long long)n * p.o_row + h * p.o_head, lane, acc);
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------
template <class Cfg>
cudaError_t launch_tree_cfg(const TreeMaps& tm, const TreeParams& p, int grid, cudaStream_t stream) {
    static std::atomic<uint64_t> attr_done{0};
    cudaError_t e = allow_smem(gsr_tree_kernel<Cfg>, Cfg::SMEM_BYTES, attr_done);
    if (e != cudaSuccess) return e;
    gsr_tree_kernel<Cfg><<<(unsigned)grid, Cfg::NUM_THREADS, Cfg::SMEM_BYTES, stream>>>(tm.q, tm.k, tm.v, p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    // the joining CTAs start while the parts' last CTAs finish, and wait for them there
    const long long rows = (long long)p.total_q * p.Hq;
    return rows >= 2048
               ? launch_early(gsr_tree_join_kernel<typename Cfg::T, Cfg::D, 1>, (unsigned)((rows + 3) / 4), kJoinThreads, 0, stream, p, grid)
               : launch_early(gsr_tree_join_kernel<typename Cfg::T, Cfg::D, 4>, (unsigned)rows, kJoinThreads, 0, stream, p, grid);
}

template <class T, int D, int NQ>
cudaError_t launch_tree_mode(const TreeMaps& tm, const TreeParams& p, int grid, cudaStream_t stream) {
    switch (score_mode(p.score)) {
        case kScorePlain: return launch_tree_cfg<TreeCfg<T, D, kScorePlain, NQ>>(tm, p, grid, stream);
        case kScoreBias: return launch_tree_cfg<TreeCfg<T, D, kScoreBias, NQ>>(tm, p, grid, stream);
        case kScoreCap: return launch_tree_cfg<TreeCfg<T, D, kScoreCap, NQ>>(tm, p, grid, stream);
        default: return launch_tree_cfg<TreeCfg<T, D, kScoreCapBias, NQ>>(tm, p, grid, stream);
    }
}

template <class T, int D>
cudaError_t launch_tree_type(const TreeMaps& tm, const TreeParams& p, int grid, cudaStream_t stream) {
    return p.nq == 1 ? launch_tree_mode<T, D, 1>(tm, p, grid, stream) : launch_tree_mode<T, D, 2>(tm, p, grid, stream);
}

}  // namespace gsr
