// llm.h - internal interface between the C-ABI layer (gsr_llm_api.cu) and the kernels of masked
// attention, tree attention over a paged cache, and the cache's bookkeeping.  Not installed; not
// part of the ABI.
#pragma once

#include "kernels.h"

namespace gsr {

// Which kernel an error word comes from, beside those of kernels.h.
enum LlmDeviceError : int {
    kDevErrKernelMaskedFwd = 0x400,
    kDevErrKernelMaskedDkv = 0x500,
    kDevErrKernelMaskedDq = 0x600,
    kDevErrKernelTree = 0x700,
};

// A (batch, head, row, D) operand: element strides, D contiguous.
struct Strided {
    void* data;
    long long batch, head, row;
};

// Which keys a query sees, and how a raw product becomes a score.  Query i of a batch row stands
// at position p = i + offset among the keys and sees one interval [lo, hi) of them (row_interval
// in attention_common.cuh).
struct MaskArgs {
    int B, Hq, Hkv, group;      // group = Hq / Hkv
    int Sq, Skv, offset;        // offset = Skv - Sq
    int causal;
    int num_docs;               // 0: no document mask
    const int* doc_bounds;      // (B, num_docs + 1)
    const int* prefix_lens;     // (B, max(num_docs, 1)) or null
};

// Scores in log2 units: y = score * log2(e).
struct ScoreArgs {
    float scale;                // softmax scale
    float sl2;                  // scale * log2(e): y = sl2 * (q.k) without a cap
    float cap_in;               // 2 log2(e) scale / cap: tanh's exponent, 0 without a cap
    float cap_z;                // (8/3) scale / cap
    float cap_out;              // cap * log2(e)
    const float* slopes;        // per query head, or null
};

struct MaskedFwdParams {
    MaskArgs mask;
    ScoreArgs score;
    Strided Q, K, V, O;
    float* lse;                 // (B, Hq, Sq) or null
    int head_group;             // item order, as in AttnParams
    int num_items;
    int splits;                 // parts of an item's keys; above 1, parts go to the workspace:
    float2* parts_ml;           // (B, Hq, splits, Sq): exponent base and sum
    float* parts;               // (B, Hq, splits, Sq, D): O, not normalised
    int* err;
    uint64_t timeout_ns;
    uint32_t test_flags;
};

// Rows of the backward pass's workspace are padded to whole 128-row tiles.
struct MaskedBwdParams {
    MaskArgs mask;
    ScoreArgs score;
    Strided dO, Q, K, V, O, dQ, dK, dV;
    const float* lse;           // (B, Hq, Sq)
    int Sp;                     // Sq rounded up to a multiple of 128
    float* offset;              // (B, Hq, Sp): row_offset less lse log2(e); -inf for rows without keys and padding
    float* neg_delta;           // (B, Hq, Sp): -rowsum(dO * O)
    // fp16 only, squares of the rows that count and are finite, else 0: |dO_i|^2 (B, Hq, Sp), the largest of 64 of
    // them (B, Hq, Sp / 64), the largest |V_j|^2 of 64 keys (B, Hkv, Skv / 64 rounded up)
    float *row_norms, *tile_norms, *v_norms;
    int q_head_group, kv_head_group;   // item order of dQ, of dK and dV: heads taken together
    int splits;                 // parts of a key tile's steps
    float* parts;               // splits > 1: (2, splits, B, Hkv, Skv, D) partial dV and dK
    int* err;
    uint64_t timeout_ns;
    uint32_t test_flags;
};

// How a cache's tensor map counts its rows in groups of 8: by page (group index page x step + row / 8,
// then the head) or by head (head x step + row / 8, then the page).
struct CacheAxes {
    bool by_head;
    int step;
};

struct TreeParams {
    int B, Hq, Hkv, group;
    int page, num_pages, table_width, max_nodes, total_q;
    ScoreArgs score;
    const void* Q;              // (total_q, Hq, D), element strides q_row, q_head
    long long q_row, q_head;
    void* O;
    long long o_row, o_head;
    Strided K, V;               // cache: batch = page stride, row = stride of a page's rows
    CacheAxes k_axes, v_axes;
    const int* table;           // (B, table_width)
    const int* kv_lens;         // (B): cached tokens, the drafted ones among them
    const int* q_starts;        // (B + 1)
    const int* parents;         // (total_q) or null: a chain
    int nq;                     // query tiles a pass
    int tile_nodes;             // nodes of a 128-row query tile: 128 / group
    int piece;                  // rows of one page copy: the page, or a part of it
    int tile_keys;              // keys of a key tile: the pieces that fit in 128 rows
    long long* unit_starts;     // workspace: (B + 1) first units, written by the first launch for the second,
    int part_rows;              // query rows of a slot
    float2* parts_ml;           // and two slots of part_rows per CTA: (m, l),
    float* parts;               // O
    int* err;
    uint64_t timeout_ns;
    uint32_t test_flags;
};

// 4-D tensor maps {D, rows, heads, batch} with 64 x 128 x 1 x 1 boxes, one per operand.
struct MaskedFwdMaps {
    CUtensorMap q, k, v;
};
// Skv == 0: no maps are read, O = 0 and lse = -inf.
cudaError_t launch_masked_fwd_f16(const MaskedFwdMaps& tm, const MaskedFwdParams& p, int D, cudaStream_t stream);
cudaError_t launch_masked_fwd_bf16(const MaskedFwdMaps& tm, const MaskedFwdParams& p, int D, cudaStream_t stream);

// Tensor maps as MaskedFwdMaps; not read where there are no queries or no keys.
struct MaskedBwdMaps {
    CUtensorMap q, k, v, dO;
};
cudaError_t launch_masked_bwd_f16_64(const MaskedBwdMaps& tm, const MaskedBwdParams& p, cudaStream_t stream);
cudaError_t launch_masked_bwd_f16_128(const MaskedBwdMaps& tm, const MaskedBwdParams& p, cudaStream_t stream);
cudaError_t launch_masked_bwd_bf16_64(const MaskedBwdMaps& tm, const MaskedBwdParams& p, cudaStream_t stream);
cudaError_t launch_masked_bwd_bf16_128(const MaskedBwdMaps& tm, const MaskedBwdParams& p, cudaStream_t stream);

// Query map {D, group, Hkv, total_q}, box {64, group, 1, tile_nodes}; cache maps {64 columns, 8 rows,
// chunks, groups of 8 rows, heads or pages}, box {64, 8, chunks, piece / 8, 1}.
struct TreeMaps {
    CUtensorMap q, k, v;
};
constexpr int kTreeMaxGrid = 160;   // CTAs at most: one per SM, bounds the workspace
cudaError_t launch_tree_f16_64(const TreeMaps& tm, const TreeParams& p, int grid, cudaStream_t stream);
cudaError_t launch_tree_f16_128(const TreeMaps& tm, const TreeParams& p, int grid, cudaStream_t stream);
cudaError_t launch_tree_bf16_64(const TreeMaps& tm, const TreeParams& p, int grid, cudaStream_t stream);
cudaError_t launch_tree_bf16_128(const TreeMaps& tm, const TreeParams& p, int grid, cudaStream_t stream);

struct TablesParams {
    int B, page, table_width, num_free, max_tokens;
    const int *kv_lens, *new_lens, *free_blocks, *free_head;
    int *table, *kv_out, *head_out, *q_starts, *positions, *slots, *counts;
};
constexpr int kTablesMaxBatch = 8192;
cudaError_t launch_block_tables(const TablesParams& p, int sms, cudaStream_t stream);

struct AppendParams {
    int N, H, D, page, num_pages;
    Strided K, V;               // new rows: row = token stride; batch unused
    Strided Kc, Vc;             // cache: batch = page stride
    const int* slots;
};
cudaError_t launch_cache_append(const AppendParams& p, int sms, cudaStream_t stream);

}  // namespace gsr
