// serving.h - internal interface between the C-ABI layer (gsr_serving_api.cu) and the kernels around
// attention: head norms with rotation, cache writes, the cache of 4 bits, drafted tokens.  Not
// installed; not part of the ABI.
#pragma once

#include <algorithm>
#include <cmath>

#include "divider.h"
#include "llm.h"

namespace gsr {

// One part of a cache of 4 bits: byte strides from page to page, head to head, row to row.
struct Bytes {
    char* data;
    long long page, head, row;
};
// Codes (D / 2 bytes a row, two values a byte, the first in the low bits) and, for each 64 values, a scale and a
// minimum of 16 bits: value = scale x code + minimum.
struct Cache4 {
    Bytes codes, params;
};

// Rows of Q and K (batch x heads x seq x D), normalised where there are weights and rotated where there is a table.
struct RopeParams {
    int B, Hq, Hkv, S, D;
    Strided Q, K, Qo, Ko;
    const void *q_weight, *k_weight;   // D values of the rows' type, or null: no norm
    const float* table;                // (rows, R): R / 2 cosines, R / 2 sines; or null: no rotation
    const int* positions;              // (B, S) or null: the row's index
    int R, rows;
    int interleaved;
    float eps;
};
cudaError_t launch_rope_fwd(const RopeParams& p, bool bf16, int sms, cudaStream_t stream);

// Gradients: Q and K are the forward's inputs, Qo and Ko the incoming gradients.
struct RopeBwdParams {
    RopeParams f;
    Strided dQ, dK;
    float *dq_weight, *dk_weight;      // D values each, where there are weights; null: not wanted
    float* parts;                      // (2, ctas, D) sums of a CTA's rows; may be null where neither is wanted
    int ctas;
};
int rope_bwd_ctas(long long batch, long long heads_q, long long heads_kv, long long seq, int D, int sms);
cudaError_t launch_rope_bwd(const RopeBwdParams& p, bool bf16, cudaStream_t stream);

// Rows of K and V to cache rows, and Q's to Qo, on the way through the same arithmetic (K and Q).
struct RopeAppendParams {
    RopeParams f;                      // B = 1, S = tokens; Ko unused
    Strided V;
    const int* slots;
    int page, num_pages;
    Strided Kc, Vc;                    // a cache of 16 bits
    Cache4 K4, V4;                     // or one of 4
};
cudaError_t launch_rope_append(const RopeAppendParams& p, bool bf16, bool four_bits, int sms, cudaStream_t stream);

struct Read4Params {
    int N, H, D, page, num_pages;
    const int* slots;
    Cache4 K4, V4;
    Strided K, V;                      // row = token stride
};
cudaError_t launch_read4(const Read4Params& p, bool bf16, cudaStream_t stream);

struct Tree4Params {
    int B, Hq, Hkv, group, D, total_q;
    int page, num_pages, table_width, max_nodes;
    ScoreArgs score;
    const void* Q;                     // (total_q, Hq, D), element strides
    long long q_row, q_head;
    void* O;
    long long o_row, o_head;
    Cache4 K, V;
    const int *table, *kv_lens, *q_starts, *parents;
    long long* unit_starts;            // workspace, where work is shared out evenly: (B + 1) first units,
    float* parts;                      // and two states a CTA
};

// How the work of attention over 4 bits is split, by sizes alone.
constexpr int kT4Warps = 4, kT4Keys = 32, kT4MaxCluster = 8;
struct Tree4Split {
    int nt, tiles;                     // column tiles of 8 query rows a CTA; row tiles a request and head
    int cluster, grid, chunks;         // CTAs that share an item (0: shared out evenly); CTAs; chunks a table's row holds
    long long starts, workspace;       // bytes
    // 16 rows at D = 64: 36 us for 41 with two (64 requests of 8 nodes over 1000 tokens); at D = 128 registers spill (209 for 187)
    static constexpr int ctas_an_sm(int nt, int D) { return nt == 1 ? 4 : D == 64 ? 3 : 2; }
    static constexpr int state_bytes(int nt, int D) { return 8 * nt * (D + 2) * 4; }
};
// A cluster an item, or all chunks shared out evenly, whichever the estimate has sooner, lengths taken as the most that
// the table holds.  A warp takes 0.9 us a chunk by itself and 2.3 us on a full SM (16 rows: 1.5 and 1.7; D = 64: 0.55 of
// it); a wave of clusters costs 5 us more, of single CTAs 4; sharing out 11 us and 4 for each item of a CTA, and with
// two items for every CTA it has nothing left to even out.  Measured, us (requests, key/value heads, tokens to;
// rows a head, D = 128), in clusters of 1, 2, 4, 8, evenly:
//   1, 8, 2000; 4       16.9  12.1   8.8   6.9   12.4        48, 8, 500; 4      11.5  17.0  21.1  37.0   18.5
//   1, 8, 32000; 4     198   103    55.4  30.9   17.7        48, 8, 2000; 4     28.3  31.7  34.6  47.7   30.0
//   4, 8, 8000; 4       53.5  31.0  18.6  15.1   18.5        48, 8, 8000; 4    100    86.3  83.7  94.2   79.5
//   16, 8, 2000; 4      17.1  14.5  14.0  18.3   18.4        256, 8, 1000; 4    59.7  82.5 120   192     76.9
//   2, 8, 4096; 160     46.8  46.2  49.6  60.6   38.4        16, 8, 4096; 160  187   229   297   433     204
//   8, 2, 1000; 16      14.8  12.5   9.8   8.6   16.8        16, 8, 4096; 64    89.6 102   121   177     88.7
inline Tree4Split tree4_split(long long B, long long Hkv, long long group, long long D, long long max_nodes, long long table_width,
                              long long page, int sms) {
    Tree4Split s{};
    s.nt = max_nodes * group > 8 ? 2 : 1;
    const long long rows = 8 * s.nt, chunks = (table_width * page + kT4Keys - 1) / kT4Keys;
    s.tiles = (int)((max_nodes * group + rows - 1) / rows);
    s.chunks = (int)chunks;
    const double items = (double)B * (double)Hkv * s.tiles, slots = (double)(Tree4Split::ctas_an_sm(s.nt, (int)D) * sms), scale = D == 64 ? 0.55 : 1.0;
    const double alone = (s.nt == 1 ? 0.9 : 1.5) * scale, full = (s.nt == 1 ? 2.3 : 1.7) * scale;
    double best = 1e30;
    for (int c = 1; c <= kT4MaxCluster; c *= 2) {
        if (c > 1 && chunks <= (long long)c / 2 * kT4Warps) break;
        const double ctas = items * c, r = ctas / slots, waves = r > 2.0 ? r + 0.3 : std::ceil(r), steps = std::ceil((double)chunks / (c * kT4Warps));
        const double t = waves * (steps * std::max(alone, full * std::pow(std::min(r, 1.0), 0.7)) + (c > 1 ? 5.0 : 4.0));
        if (t < best) {
            best = t;
            s.cluster = c;
            s.grid = (int)ctas;
        }
    }
    if (items < 2 * slots && 11.0 + 4.0 * items / slots + items * (double)chunks * full / (slots * kT4Warps) < best) {
        s.cluster = 0;
        s.grid = (int)slots;
        s.starts = ((B + 1) * 8 + 255) / 256 * 256;
        s.workspace = s.starts + 2ll * s.grid * Tree4Split::state_bytes(s.nt, (int)D);
    }
    return s;
}
cudaError_t launch_tree4_f16(const Tree4Params& p, const Tree4Split& split, cudaStream_t stream);
cudaError_t launch_tree4_bf16(const Tree4Params& p, const Tree4Split& split, cudaStream_t stream);

struct VerifyParams {
    int B, N, V, max_nodes;
    const float *target, *draft;       // (N, V) rows target_row, draft_row apart; draft may be null
    long long target_row, draft_row;
    const int *tokens, *q_starts, *parents;
    const float *u_accept, *u_sample;
    int *path, *counts, *next;
};
cudaError_t launch_verify(const VerifyParams& p, cudaStream_t stream);

}  // namespace gsr
