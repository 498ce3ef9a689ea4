// serving.h - internal interface between the C-ABI layer (gsr_serving_api.cu) and the kernels around
// attention: head norms with rotation, cache writes, the cache of 4 bits, drafted tokens.  Not
// installed; not part of the ABI.
#pragma once

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
    float *dq_weight, *dk_weight;      // D values each, where there are weights
    float* parts;                      // (2, ctas, D) sums of a CTA's rows
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
};
cudaError_t launch_tree4_f16(const Tree4Params& p, int sms, cudaStream_t stream);
cudaError_t launch_tree4_bf16(const Tree4Params& p, int sms, cudaStream_t stream);

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
