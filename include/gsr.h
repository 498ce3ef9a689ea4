/*
 * gsr.h - fused GEMM + scale + ReLU on GB300 (sm_103a):
 *
 *     C[m,n] = ReLU( alpha * sum_{k=0}^{K-1} A[m,k] * B[k,n] )
 *
 * Operator definition: "Tutorial14: 使用TileLang语言编写attention算子" (PKUHPC
 * scow-tutorial), section 3 (算子介绍) gives the formula and ReLU(x) = max(x, 0);
 * section 2 (编写算子), the gemm_fused kernel, fixes the data types (A, B, C
 * float16, accumulator float32, scale float32) and the order of the epilogue
 * (multiply by the scale first, then the max with 0, then the fp16 store).
 *
 * Plain C ABI: pointers and sizes only.  Every entry point returns a
 * gsr_status and never aborts the process.  Entry points that launch work are
 * asynchronous on the given stream: returning GSR_OK means the work was
 * queued, not that it finished.  A NULL stream is the legacy default stream.
 * Thread-safety: the entry points may be called from several host threads.
 */
#ifndef GSR_H_
#define GSR_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t / CUstream; declared here so this header needs no
 * CUDA header. */
struct CUstream_st;

typedef enum gsr_status {
    GSR_OK = 0,
    /* A negative size, a size above 2^31 - 1, a NULL pointer where data is
     * needed, or a NULL stream pointer argument where one is required. */
    GSR_ERR_INVALID_ARG = 1,
    /* A, B or C not 16-byte aligned, or N or K not a multiple of 8 (the tensor
     * copy engine needs every row pitch to be a multiple of 16 bytes). */
    GSR_ERR_ALIGNMENT = 2,
    /* C overlaps A or B. */
    GSR_ERR_ALIAS = 3,
    /* A CUDA runtime call failed; gsr_last_cuda_error() has its code. */
    GSR_ERR_CUDA = 4,
    /* A kernel gave up on a bounded wait (reported by gsr_device_status). */
    GSR_ERR_DEVICE_TIMEOUT = 5,
    /* The current device is not compute capability 10.3 (GB300). */
    GSR_ERR_UNSUPPORTED_DEVICE = 6,
    /* gemm_scale_relu_noalloc: these sizes need more scratch than its fixed
     * array holds. */
    GSR_ERR_SCRATCH_LIMIT = 7
} gsr_status;

/*
 * C = ReLU(alpha * A.B).
 *
 *   A      device pointer, M x K float16, row-major (row stride K elements).
 *   B      device pointer, K x N float16, row-major (row stride N elements).
 *   C      device pointer, M x N float16, row-major (row stride N elements);
 *          written, never read.  Must not overlap A or B.
 *   M,N,K  sizes, 0 <= M, N, K <= 2^31 - 1; N and K multiples of 8.
 *   alpha  float32 scale, applied to the float32 sum before the ReLU.
 *   stream CUDA stream the work is queued on (NULL: legacy default stream).
 *
 * All three buffers are owned by the caller and must stay valid until the
 * work on `stream` has finished.  Results: the sum is carried in float32 on
 * the tensor cores and rounded once to float16 (nearest, ties to even).
 * ReLU of -0 or NaN gives 0.  M == 0 or N == 0: nothing to do, GSR_OK.
 * K == 0: C is filled with zeros (ReLU(alpha * 0)).
 *
 * Paths: M <= 64 runs the small-M kernel (B streamed once, K split across
 * SMs) when B holds at least 16 MiB, and so do 65 to 128 rows when B is large and
 * the tiles below would leave SMs idle; larger M runs a tiled kernel, on CTA pairs with 256 x 256 tiles when
 * there are enough of them to fill the GPU (or K is long), else one CTA per
 * 128-row tile (gsr_select_path gives the rules).
 *
 * Device memory the library owns: on the first call on each (device, stream)
 * pair it allocates 16 bytes for that stream (the kernels' error word and the
 * attention kernel's work counters), and the small-M kernel keeps fp32 partial
 * tiles and per-tile ticket counters in a workspace allocated (or grown) on the
 * first small-M call on the pair.  Both stay until gsr_release_stream() for that
 * stream or gsr_shutdown().  Calls on different streams never share them; such a
 * first call synchronises its stream and so should not be made during stream
 * capture.  Once a stream has seen a call of the same kind (and size, for the
 * small-M workspace), further calls on it only encode tensor maps on the host
 * and launch, so they can be captured into a CUDA graph and replayed; a
 * replay reads whatever the captured buffers hold then.  A captured call keeps
 * using the capture stream's library memory (error word, attention work
 * counters, small-M workspace): replays must not run at the same time as each
 * other or as other library calls on that stream.  The per-thread default stream
 * (cudaStreamPerThread) is a stream of each calling thread's, with library memory of
 * its own; a thread that ends calls gsr_release_stream for it first, or its memory
 * stays until gsr_shutdown().
 */
gsr_status gemm_scale_relu(const void* A, const void* B, void* C, int64_t M, int64_t N,
                           int64_t K, float alpha, struct CUstream_st* stream);

/*
 * C = alpha * A.B, the same GEMM without the ReLU; alpha = 1 gives the plain
 * tiled matrix product.  ("TileLang: создание высокопроизводительных GPU-ядер"
 * survey page, section 2 "Тилированное умножение матриц": make_matmul, the plain
 * tiled tensor-core GEMM the fused operator extends.)  Arguments, layout,
 * ownership, paths and errors as for gemm_scale_relu; K == 0 gives zeros.
 */
gsr_status gemm_scale(const void* A, const void* B, void* C, int64_t M, int64_t N, int64_t K,
                      float alpha, struct CUstream_st* stream);

/*
 * C[m,n] = GELU( sum_k A[m,k] * B[k,n] + bias[n] ), GELU in its tanh form
 * 0.5 x (1 + tanh( sqrt(2/pi) (x + 0.044715 x^3) )), computed in fp32 on the
 * accumulator before the fp16 store.  (Same survey page, section 4 "Слияние
 * эпиколов: GEMM + Bias + GELU": make_matmul_bias_gelu adds the bias and applies
 * an exponential-formula GELU approximation in registers.)
 *
 *   bias   device pointer to N float16 values, 16-byte aligned, must not
 *          overlap C; read, never written.
 * Other arguments, paths and errors as for gemm_scale_relu.  K == 0 gives
 * C[m,n] = GELU(bias[n]).
 */
gsr_status gemm_bias_gelu(const void* A, const void* B, const void* bias, void* C, int64_t M,
                          int64_t N, int64_t K, struct CUstream_st* stream);

/*
 * Attention forward, FlashAttention style:
 *
 *     O = softmax( softmax_scale * Q K^T  [causal mask] ) V        per batch and head
 *
 * (aikraft.ru TileLang tutorial survey "TileLang: создание высокопроизводительных
 * GPU-ядер", section 6 "FlashAttention: Слияние внимания": online softmax with running
 * maxima, normalisation sums and rescaling factors, causal masks, pipelined copies.)
 *
 *   Q      device pointer, (batch, heads, seq_q, head_dim) float16, row-major.
 *   K, V   device pointers, (batch, heads, seq_kv, head_dim) float16, row-major.
 *   O      device pointer, (batch, heads, seq_q, head_dim) float16; written.
 *   lse    optional device pointer (NULL: not written), (batch, heads, seq_q) float32:
 *          the natural-log log-sum-exp of each query's scaled, masked scores.
 *   head_dim        64 or 128.
 *   softmax_scale   0 selects 1/sqrt(head_dim).
 *   causal          nonzero: query i keeps key j only when j <= i + (seq_kv - seq_q)
 *                   (lower triangle aligned to the bottom-right corner).
 * Scores and softmax in fp32, P rounded to fp16 for the second product, output rounded
 * once to fp16.  masked_attention_fwd below computes the same and more, faster (4 x 32 x 4096 x
 * 128 causal 457 us, this call 537).  A query with no key left (causal with seq_q > seq_kv, or seq_kv == 0)
 * gets O = 0 and lse = -inf.  All pointers 16-byte aligned (lse 4-byte); O and lse must
 * not overlap the inputs or each other.  Caller-owned buffers; asynchronous on `stream`;
 * errors as for gemm_scale_relu.
 */
gsr_status flash_attention_fwd(const void* Q, const void* K, const void* V, void* O, float* lse,
                               int64_t batch, int64_t heads, int64_t seq_q, int64_t seq_kv,
                               int64_t head_dim, float softmax_scale, int causal,
                               struct CUstream_st* stream);

/* ------------------------------------------------------------------------------------------
 * Attention of language models: masked attention with its gradient, a paged key/value cache, and
 * attention of drafted tokens over it.  float16 or bfloat16, head_dim 64 or 128, any number of
 * query heads per key/value head.  Scores, softmax and sums in float32.  Caller-owned buffers;
 * asynchronous on `stream`; with workspaces of their own, calls and graph replays share no memory
 * but the error word and may run at the same time on different streams.
 * ------------------------------------------------------------------------------------------ */
typedef enum gsr_dtype { GSR_F16 = 0, GSR_BF16 = 1 } gsr_dtype;

/*
 * A batch x head x row x D operand: element strides, multiples of 8, D contiguous, data 16-byte
 * aligned.  Any order of the other three dimensions is fine (batch, row, head as a projection
 * leaves it; the parts of a fused projection's output).  A dimension of size 1 has no stride; a
 * stride of 0 (a broadcast) is refused with GSR_ERR_INVALID_ARG.  An output must share no element with
 * an input or another output (GSR_ERR_ALIAS): views with the same strides are compared element by
 * element, so the parts of one buffer may lie in any order; views whose strides differ must not meet
 * from their first to their last byte.
 */
typedef struct gsr_tensor {
    void* data;
    int64_t stride_batch, stride_head, stride_row;
} gsr_tensor;

/*
 * Sizes, masks and scores of masked attention.  Query i stands at position p = i + (seq_kv -
 * seq_q) among the keys; query head h reads key/value head h / (heads_q / heads_kv).
 *
 *   score(i, j) = s - slope[h] |p - j|,   s = softmax_scale q_i.k_j without a cap, else
 *                                         s = softcap tanh(softmax_scale q_i.k_j / softcap)
 *
 * Keys a query sees: those of its document [start, end) (all of them without documents), cut with
 * `causal` to j <= p or j < start + prefix, whichever reaches further.
 *
 *   softmax_scale  0 selects 1/sqrt(head_dim).
 *   softcap        0: no cap; else 0 < softcap <= 1024 (a capped score is off by about softcap 2^-23).
 *   alibi_slopes   NULL: no distance bias; else device pointer to heads_q float32.  Constants: no
 *                  gradient is computed for them.
 *   doc_bounds     NULL: no documents; else device pointer to batch x (num_docs + 1) int32,
 *                  ascending within a batch row: document d of row b holds positions
 *                  [doc_bounds[b][d], doc_bounds[b][d + 1]).  Positions outside all documents are
 *                  padding: they see nothing and nothing sees them, whatever they hold (NaN too).
 *                  Equal boundaries are an empty document.  Needs seq_q == seq_kv.  Boundaries
 *                  that are not ascending give unspecified results, without a fault.
 *   prefix_lens    NULL: none; else device pointer to batch x max(num_docs, 1) int32, the number
 *                  of leading keys of each document (or row) that all its queries see.  Needs
 *                  `causal`.
 */
typedef struct gsr_attention_desc {
    int64_t batch, heads_q, heads_kv, seq_q, seq_kv, head_dim;
    int32_t dtype; /* gsr_dtype */
    int32_t causal;
    float softmax_scale;
    float softcap;
    const float* alibi_slopes;
    const int32_t* doc_bounds;
    int64_t num_docs;
    const int32_t* prefix_lens;
} gsr_attention_desc;

/*
 * O = softmax(score) V over the keys each query sees.  Q, O: batch x heads_q x seq_q x head_dim;
 * K, V: batch x heads_kv x seq_kv x head_dim; lse: batch x heads_q x seq_q float32, contiguous
 * (NULL: not written), the natural log-sum-exp of the scores.  A query that sees no key gets O = 0
 * and lse = -inf.  Keys a query does not see have no influence on it, also when they hold
 * infinities or NaN.  An infinity or NaN in V makes its column infinite or NaN for every query that
 * sees the key, however small the probability, and leaves the other columns and lse as they are; the
 * time of a call grows little with them.  Probabilities are rounded to the operands' type for the second product, the
 * output once.  O must share no element with an input, lse lies apart from everything.
 *
 *   workspace  device pointer, 16-byte aligned, masked_attention_fwd_workspace(desc) bytes (0 where
 *              there are queries enough for the SMs; it depends on the sizes alone), for this call
 *              alone until it has finished; or NULL: where one is needed, one that the library keeps for
 *              the stream (grown after a wait for the stream; released by gsr_release_stream).  In a
 *              stream capture NULL then gives GSR_ERR_INVALID_ARG: a graph has a workspace of its own.
 */
int64_t masked_attention_fwd_workspace(const gsr_attention_desc* desc);
gsr_status masked_attention_fwd(const gsr_attention_desc* desc, const gsr_tensor* Q, const gsr_tensor* K,
                                const gsr_tensor* V, const gsr_tensor* O, float* lse, void* workspace,
                                int64_t workspace_bytes, struct CUstream_st* stream);

/*
 * Gradients of masked_attention_fwd: dQ, dK, dV from dO and the forward's inputs, O and lse (dO,
 * O, dQ shaped as Q; dK, dV as K).  dK and dV sum over the query heads of a group.  Results do not
 * depend on the order of execution.  P and dS are rounded to the operands' type for the matrix
 * products; in float16 dS carries powers of two, one for each query in dQ and one for each key in dK (the
 * same for nearby keys of a document), that keep it in range whatever the size of dO there.  They take
 * V's size by key/value head: values 2^13 below the largest of their head lose digits of dS.
 * Queries without keys get dQ = 0 and add nothing, whatever their dO holds.  Infinities and NaN in
 * dO, Q, K and V reach the gradients of the pairs that see each other and no other elements, and a call
 * with them takes about as long as one without.
 *
 *   workspace  masked_attention_bwd_workspace(desc) bytes, as for masked_attention_fwd.
 */
int64_t masked_attention_bwd_workspace(const gsr_attention_desc* desc);
gsr_status masked_attention_bwd(const gsr_attention_desc* desc, const gsr_tensor* dO, const gsr_tensor* Q,
                                const gsr_tensor* K, const gsr_tensor* V, const gsr_tensor* O,
                                const float* lse, const gsr_tensor* dQ, const gsr_tensor* dK,
                                const gsr_tensor* dV, void* workspace, int64_t workspace_bytes,
                                struct CUstream_st* stream);

/*
 * Attention of drafted tokens over a paged cache.  Request b has kv_lens[b] tokens in the cache;
 * the last T_b = q_starts[b + 1] - q_starts[b] of them are its drafted tokens, whose keys and
 * values have been written like any other token's.  They are the nodes of a tree: row q_starts[b]
 * + t of Q and O belongs to node t, parents[q_starts[b] + t] is the node above it (an earlier one,
 * or -1 for the token before the tree).  A node sees every token before the tree, its ancestors
 * and itself, and stands at position kv_lens[b] - T_b + its depth.  parents == NULL: a chain (each
 * node below the one before it).  T_b = 1 is an ordinary decoding step; T_b = 0 is fine.
 *
 *   k_cache, v_cache  num_pages pages of page_size rows (a multiple of 8; stride_batch steps from
 *                     page to page, and it or else stride_head is a multiple of 8 stride_row, as in
 *                     every dense layout); row r of request b is row r % page_size of page
 *                     block_tables[b][r / page_size].  Entries outside [0, num_pages) hold no
 *                     tokens: nothing sees them.  Cache rows behind kv_lens[b] have no influence.
 *   block_tables      batch x table_width int32.  Lengths above table_width x page_size are cut.
 *   max_nodes         the most nodes of a request, 1 to GSR_TREE_MAX_NODES.  Rows of further
 *                     nodes and rows behind q_starts[batch] are left as they were.
 *   softcap, alibi_slopes, softmax_scale  as in gsr_attention_desc.
 *   Q, O              total_q x heads_q x head_dim with the given strides; heads_q / heads_kv <= 128.
 * kv_lens, q_starts (batch + 1), parents (total_q): device int32.  A node that sees nothing gets
 * O = 0.  Infinities and NaN in V reach their columns of the nodes that see them, as in
 * masked_attention_fwd, and no sibling.
 *
 *   workspace  device pointer, 16-byte aligned, tree_attention_workspace(desc) bytes, for this
 *              call alone until it has finished; or NULL, as for masked_attention_fwd.
 */
#define GSR_TREE_MAX_NODES 64
typedef struct gsr_tree_desc {
    int64_t batch, total_q, heads_q, heads_kv, head_dim;
    int64_t num_pages, page_size, table_width, max_nodes;
    int64_t q_stride_row, q_stride_head, o_stride_row, o_stride_head;
    int32_t dtype; /* gsr_dtype */
    float softmax_scale;
    float softcap;
    const float* alibi_slopes;
} gsr_tree_desc;
int64_t tree_attention_workspace(const gsr_tree_desc* desc);
gsr_status tree_attention_fwd(const gsr_tree_desc* desc, const void* Q, const gsr_tensor* k_cache,
                              const gsr_tensor* v_cache, const int32_t* block_tables, const int32_t* kv_lens,
                              const int32_t* q_starts, const int32_t* parents, void* O, void* workspace,
                              int64_t workspace_bytes, struct CUstream_st* stream);

/*
 * One step's bookkeeping of a paged cache, on the device: request b has kv_lens[b] tokens and gets
 * new_lens[b] more (negative lengths count as 0).  Pages are taken from free_blocks, from entry
 * free_head[0] on, in request order.
 *
 *   block_tables   batch x table_width, updated in place: the new pages' entries are written.
 *   kv_lens_out    batch: kv_lens + new_lens.           free_head_out  1: free_head + pages taken.
 *   q_starts       batch + 1: where each request's new tokens start among all of them.
 *   positions, slots  max_tokens: each new token's position in its request and its row in the
 *                  cache, page x page_size + row; -1 behind the last token.  Positions count tokens as they
 *                  are stored, kv_lens + index: a prompt's or a chain's.  Nodes of a tree that branches stand
 *                  elsewhere, at kv_lens + depth (see tree_attention_fwd).
 *   counts         3: new tokens, pages taken, pages missing.
 * Pages are missing when the free list ends or a request outgrows table_width; their table
 * entries (those inside the table) and their tokens' slots are -1.  All int32 device arrays;
 * outputs overlap nothing (kv_lens_out and free_head_out are not the inputs: swap them between
 * steps).  batch <= 8192; the sum of new_lens and num_pages x page_size below 2^31.
 */
gsr_status kv_block_tables(const int32_t* kv_lens, const int32_t* new_lens, const int32_t* free_blocks,
                           const int32_t* free_head, int32_t* block_tables, int32_t* kv_lens_out,
                           int32_t* free_head_out, int32_t* q_starts, int32_t* positions, int32_t* slots,
                           int32_t* counts, int64_t batch, int64_t table_width, int64_t page_size,
                           int64_t num_free, int64_t max_tokens, struct CUstream_st* stream);

/*
 * Writes new keys and values to their cache rows: row n of K (V) goes to row slots[n] % page_size
 * of page slots[n] / page_size.  Slots outside the cache (-1: padding) are skipped; other cache
 * rows are left as they were.  K, V: tokens x heads x head_dim (stride_row steps from token to
 * token; stride_batch unused) of any 16-bit type, head_dim a multiple of 8.  Where two tokens have
 * the same slot, the row holds pieces of either.  k_cache and v_cache may be views of one buffer
 * that share no element, as outputs of gsr_tensor's description (else GSR_ERR_ALIAS).
 */
gsr_status kv_cache_append(const gsr_tensor* K, const gsr_tensor* V, const int32_t* slots,
                           const gsr_tensor* k_cache, const gsr_tensor* v_cache, int64_t tokens,
                           int64_t heads, int64_t head_dim, int64_t num_pages, int64_t page_size,
                           struct CUstream_st* stream);

/* ------------------------------------------------------------------------------------------
 * Before and after attention: head norms with the position rotation, cache writes with both on the
 * way, a cache of 4 bits, and which drafted tokens to keep.  Types, strides and streams as above;
 * arithmetic in float32, each result rounded once.
 * ------------------------------------------------------------------------------------------ */

/*
 * Rows x of D values:  y = rot(x w / sqrt(mean(x^2) + eps)).
 *
 *   q_weight, k_weight  NULL: rows of Q (K) are not normalised; else device pointer to head_dim
 *                  values of the rows' type, 16-byte aligned.
 *   cos_sin        NULL: no rotation; else device pointer to table_rows x rotary_dim float32, 16-byte
 *                  aligned: a position's rotary_dim / 2 cosines, then as many sines.  Pair i of the
 *                  first rotary_dim columns (a multiple of 16, 16 to head_dim) turns to
 *                  (a cos_i - b sin_i, b cos_i + a sin_i); the other columns stay.
 *   interleaved    0: pair i is columns i and i + rotary_dim / 2; else 2 i and 2 i + 1.
 *   positions      device pointer to batch x seq int32, a row of the table for each token; NULL: a
 *                  token's index in its row (seq <= table_rows).  Not read without cos_sin.  A negative
 *                  one marks padding: its rows are 0.  One behind the table makes the rows NaN.
 *   eps            >= 0, finite.
 */
typedef struct gsr_rope_desc {
    int64_t batch, heads_q, heads_kv, seq, head_dim, rotary_dim, table_rows;
    int32_t dtype; /* gsr_dtype */
    int32_t interleaved;
    float eps;
    const void* q_weight;
    const void* k_weight;
    const float* cos_sin;
    const int32_t* positions;
} gsr_rope_desc;

/*
 * Q_out = y(Q), K_out = y(K).  Q, Q_out: batch x heads_q x seq x head_dim; K, K_out with heads_kv
 * heads.  heads_q or heads_kv may be 0 (its operands are then not looked at).  An output may be the
 * very view of its input (a call in place); otherwise outputs share no element with anything.
 */
gsr_status qk_norm_rope_fwd(const gsr_rope_desc* desc, const gsr_tensor* Q, const gsr_tensor* K,
                            const gsr_tensor* Q_out, const gsr_tensor* K_out, struct CUstream_st* stream);

/*
 * Gradients dQ, dK and, where there are weights, dq_weight, dk_weight (head_dim float32 each, written,
 * not added to) from dQ_out, dK_out and the forward's inputs Q, K (each read only where there is a
 * weight).  A weight whose operand has no heads gets a gradient of 0, or none (NULL).  dQ may be the very
 * view of dQ_out or of Q, dK likewise.  Padding's gradients are 0 and
 * it adds nothing to the weights', whatever its rows hold.  Results do not depend on the order of
 * execution.
 *
 *   workspace  qk_norm_rope_bwd_workspace(desc) bytes, or NULL, as for masked_attention_fwd.
 */
int64_t qk_norm_rope_bwd_workspace(const gsr_rope_desc* desc);
gsr_status qk_norm_rope_bwd(const gsr_rope_desc* desc, const gsr_tensor* dQ_out, const gsr_tensor* dK_out,
                            const gsr_tensor* Q, const gsr_tensor* K, const gsr_tensor* dQ, const gsr_tensor* dK,
                            float* dq_weight, float* dk_weight, void* workspace, int64_t workspace_bytes,
                            struct CUstream_st* stream);

/*
 * kv_cache_append with the norm and rotation on the way: row n of y(K) and of V goes to cache row
 * slots[n], and Q_out = y(Q) where heads_q > 0 (in place or apart, as in qk_norm_rope_fwd).  desc: batch
 * 1, seq tokens; cos_sin needs positions.  Those of prompts, chains and single tokens are
 * kv_block_tables'; a node of a tree that branches stands at the tokens before the tree + its depth, as
 * tree_attention_fwd has it, so that siblings are turned alike and a kept path is turned as the chain that it
 * becomes.  Slots outside the cache and tokens of negative position are skipped; other cache rows are left as they
 * were.  Caches as in kv_cache_append; no two tokens of a call have the same slot (the row would hold pieces of both).
 */
gsr_status kv_cache_append_rope(const gsr_rope_desc* desc, const gsr_tensor* Q, const gsr_tensor* K,
                                const gsr_tensor* V, const int32_t* slots, const gsr_tensor* Q_out,
                                const gsr_tensor* k_cache, const gsr_tensor* v_cache, int64_t num_pages,
                                int64_t page_size, struct CUstream_st* stream);

/*
 * A cache of 4 bits a value: each 64 values of a row have a scale s and a minimum m, both of the
 * rows' 16-bit type, and a value is s c + m with a code c of 0 to 15: 4.5 bits a value.
 *
 *   codes   page x head x row of head_dim / 2 bytes, value 2 i in byte i's low half, 2 i + 1 in its
 *           high half.  Strides in bytes, multiples of 16, data 16-byte aligned.
 *   params  page x head x row of head_dim / 64 pairs (s, m).  Strides in 16-bit elements, multiples of
 *           head_dim / 32, data aligned to head_dim / 16 bytes.
 * Rows of a head that lie together (pages, heads, rows) are read fastest.  Dimensions and overlaps
 * as in gsr_tensor; codes and params lie in buffers of their own.
 */
typedef struct gsr_cache4 {
    gsr_tensor codes, params;
} gsr_cache4;

/*
 * kv_cache_append_rope into caches of 4 bits: m is the least of 64 values, s = (largest - m) / 15 (both
 * rounded to the rows' type), c = (x - m) / s rounded to the nearest even and cut to 0..15, 0 where s is
 * 0.  64 values that hold an infinity or NaN, span more than a float32, or whose minimum or scale is beyond the
 * rows' type (keys after their norm or rotation) become NaN.
 */
gsr_status kv_cache4_append_rope(const gsr_rope_desc* desc, const gsr_tensor* Q, const gsr_tensor* K,
                                 const gsr_tensor* V, const int32_t* slots, const gsr_tensor* Q_out,
                                 const gsr_cache4* k_cache, const gsr_cache4* v_cache, int64_t num_pages,
                                 int64_t page_size, struct CUstream_st* stream);

/*
 * Rows of caches of 4 bits as 16-bit values, for a prompt that attends to what is cached: row n of K
 * (V), tokens x heads x head_dim, is cache row slots[n]; rows of slots outside the cache are left as
 * they were.
 */
gsr_status kv_cache4_read(const gsr_cache4* k_cache, const gsr_cache4* v_cache, const int32_t* slots,
                          const gsr_tensor* K, const gsr_tensor* V, int64_t tokens, int64_t heads,
                          int64_t head_dim, int64_t num_pages, int64_t page_size, int32_t dtype,
                          struct CUstream_st* stream);

/*
 * tree_attention_fwd over caches of 4 bits (desc->dtype: that of Q, O and the scales; alibi_slopes
 * NULL; page and row strides below 2^32 bytes).  p s is rounded to float16, whatever the type, for the
 * second product (p to float32 for the minima); where the scales of one row of V are 2^20
 * apart, the smaller one's columns lose digits.  A query's values 2^25 below its largest lose digits, and
 * bfloat16 queries that reach 2^112 get NaN.  Scales are not negative.  A NaN scale or minimum in V makes
 * its 64 columns NaN for the nodes that see the key, in K all columns, and has no influence on other nodes.
 *
 *   workspace  tree_attention4_workspace(desc) bytes (0 where there is little work; it depends on the sizes
 *              alone), or NULL, as for masked_attention_fwd.
 */
int64_t tree_attention4_workspace(const gsr_tree_desc* desc);
gsr_status tree_attention4_fwd(const gsr_tree_desc* desc, const void* Q, const gsr_cache4* k_cache,
                               const gsr_cache4* v_cache, const int32_t* block_tables, const int32_t* kv_lens,
                               const int32_t* q_starts, const int32_t* parents, void* O, void* workspace,
                               int64_t workspace_bytes, struct CUstream_st* stream);

/*
 * Which drafted tokens the target's probabilities keep, from given random numbers, and the token that
 * follows.  Nodes as in tree_attention_fwd, but node 0 of a request is the last token that is already
 * decided, and the drafts hang below it: node t > 0 is the draft draft_tokens[q_starts[b] + t] for the
 * place after its parent (an earlier node; parents == NULL: a chain).  Nodes that do not hang below node 0
 * are not reached.  Row q_starts[b] + t of target_probs is the target's distribution after node t, row
 * q_starts[b] + t of draft_probs the one that node t's token was drawn from; draft_probs == NULL:
 * tokens were not drawn (retrieved, or a head's best guesses).
 *
 * From node 0 on, children are tried in their order: with r = p, the target's row, and T = 1, child c with
 * token x is kept if u_accept[c] T q(x) < r(x); else r = max(r - T q, 0), T = sum(r), and the next child is
 * tried.  Without draft_probs q(x) is 1, and a refusal takes x out of r and its r(x) off T.  Below a kept
 * child the same goes on with its row.  Where no child is kept (or there is none) the next token is the
 * first v with r(0) + ... + r(v) > u_sample[b] sum(r), its last node's row in place of an r of zeros (-1
 * if that is zero too).  Tokens are then distributed as the target's own.
 *
 *   target_probs, draft_probs  total_q x vocab float32, rows target_stride_row (draft_stride_row)
 *                  elements apart; vocab up to 2^24.  NaN counts as 0, other values are cut to 0..1.
 *   u_accept       total_q float32 in [0, 1).      u_sample  batch float32 in [0, 1).
 *   path           batch x max_nodes int32: the kept drafts' nodes from the root on, then -1.
 *   counts         batch int32: how many.          next_tokens  batch int32.
 * Kept nodes' cache rows lie where the tree was written.  Before the next step the caller moves them together, in
 * K and V: row L + path[i] of the request to row L + 1 + i, L tokens before node 0.  Rows of 4 bits are moved as codes
 * and params (read and written again they would get other codes).
 *
 * A request without nodes gets 0 and -1.  Nodes behind max_nodes (at most GSR_TREE_MAX_NODES) are not
 * tried.  Tokens outside the vocabulary are refused.  Sums are exact in fixed point, 45 bits behind the
 * point: results are the same on every run (a row's sum, 1 of a distribution, must stay below 2^18).
 */
typedef struct gsr_verify_desc {
    int64_t batch, total_q, vocab, max_nodes, target_stride_row, draft_stride_row;
} gsr_verify_desc;
gsr_status verify_drafts(const gsr_verify_desc* desc, const float* target_probs, const float* draft_probs,
                         const int32_t* draft_tokens, const int32_t* q_starts, const int32_t* parents,
                         const float* u_accept, const float* u_sample, int32_t* path, int32_t* counts,
                         int32_t* next_tokens, struct CUstream_st* stream);

/*
 * gemm_scale_relu with the operands in host memory: copies A and B host ->
 * device into the caller's device buffers dA and dB, runs gemm_scale_relu
 * into dC and copies C back device -> host, all ordered on `stream`: the call
 * starts after the work already queued there, and work queued after it sees hC
 * complete.  The host buffers should be page-locked (cudaHostAlloc / pinned) for
 * the copies to be asynchronous.  Sizes, alignment and errors as for
 * gemm_scale_relu; dC must not overlap dA or dB.
 * From 2^33 flop (~8.6 GFLOP) and 1024 rows up the three parts overlap: A is copied
 * in 2..8 chunks of rows, and B whole or, where C has more elements than A and B
 * together, in 2..4 blocks of columns (each a multiple of 256 columns, wide enough
 * for a full wave of the CTA-pair kernel); the product of each chunk of rows and
 * block of columns runs on `stream` as soon as both have landed, and that block of
 * C goes back (a strided copy) while later ones are copied in.  dB and dC then
 * hold the whole matrices as for gemm_scale_relu; only the order in which their
 * parts are written changes.  The copies run on two library-owned streams per device (one
 * per direction, joined to `stream` by library-owned events; created on first
 * use, released by gsr_shutdown), and concurrent calls on one device queue their
 * copies one call after the other.
 */
gsr_status gemm_scale_relu_host(const void* hA, const void* hB, void* hC, void* dA, void* dB,
                                void* dC, int64_t M, int64_t N, int64_t K, float alpha,
                                struct CUstream_st* stream);

/*
 * gemm_scale_relu without any device-memory allocation, for callers that cannot
 * let a library allocate: for example a serving runtime that plans all of its
 * device memory at start-up and forbids allocations afterwards, or a
 * latency-critical loop that cannot take the implicit synchronisation of a
 * first-time cudaMalloc.  (No counterpart on the pages: they allocate through
 * the TileLang JIT and PyTorch.)
 *
 * Arguments, layout, ownership and result are those of gemm_scale_relu, for
 * the small-M kernel only: 1 <= M <= 64 (M > 64 returns GSR_ERR_INVALID_ARG;
 * M == 0 or N == 0 is a no-op and K == 0 clears C, as there).  The small-M kernel
 * has no raster order to set: gsr_set_raster_group does not apply to it.  The caller
 * passes A, B and C; the kernel's scratch (error word, per-tile tickets and
 * split-K partial tiles) lives in one fixed 12 MiB array inside the library,
 * which every GPU that loads the library holds until the process exits.
 * Sizes whose scratch would not fit return GSR_ERR_SCRATCH_LIMIT before any
 * work is queued; on a 152-SM GB300 that happens only for N above about 4.0e8
 * (sizes whose per-tile tickets alone cannot fit are refused before any CUDA
 * call).  The call never runs cudaMalloc, cudaFree or any other allocating
 * routine.
 *
 * Set-up: the first call on each device, with that device current, looks up the
 * array's device address and makes the kernel variants resident.  Under CUDA's
 * default lazy module loading, that is when the driver places the array and the
 * kernels' code on the device: an allocation by the driver, which can also
 * synchronise.  A caller with a fixed memory plan should therefore make one call
 * on each device during start-up.  Later calls place nothing.
 *
 * Every call shares the array and it keeps the last call's contents; each call
 * clears the parts that must start at zero, on `stream`, before its kernel.
 * Calls whose work overlaps on the GPU (for example on two streams with no
 * ordering between them) race on the array and produce wrong results: order
 * them on one stream.  If a bounded wait inside the kernel runs out, C is left
 * unspecified; gsr_device_status reports GSR_ERR_DEVICE_TIMEOUT for the most
 * recent call of this entry point on the current device, until it has been read
 * once or the next call starts.  It reads the word after the work of the stream it
 * is given: pass the stream the call was queued on (or one ordered after it).
 */
gsr_status gemm_scale_relu_noalloc(const void* A, const void* B, void* C, int64_t M, int64_t N,
                                   int64_t K, float alpha, struct CUstream_st* stream);

/*
 * Waits for `stream`, then reads and clears the error word of the (current
 * device, stream) pair, and that of gemm_scale_relu_noalloc on the current device.
 * Returns GSR_ERR_DEVICE_TIMEOUT if a kernel queued on that stream since the last
 * call (or the latest gemm_scale_relu_noalloc call on the device) gave up on a
 * bounded wait, GSR_ERR_CUDA if the stream reported an error, else GSR_OK.  The
 * output of the call that gave up is unspecified; later calls are correct
 * whether or not this function is called (the small-M kernel leaves its ticket
 * counters at zero even when it gives up).  `code` (may be NULL) receives the raw
 * device error code, 0 if none: low byte = which wait gave up (1 producer
 * waiting for a free stage, 2 MMA issuer waiting for loaded data, 3 MMA issuer
 * waiting for a free accumulator, 4 epilogue waiting for a finished
 * accumulator, 5 teardown drain, 6 shared-memory window not 1024-byte aligned:
 * the kernel returned at once), 0x100 = tiled kernel, 0x200 = small-M,
 * 0x300 = attention, 0x400 = masked attention, 0x500 and 0x600 = its gradients of K, V and of Q,
 * 0x700 = tree attention.
 */
gsr_status gsr_device_status(struct CUstream_st* stream, int* code);

/*
 * Releases the library's state for the (current device, stream) pair: the
 * stream's 16 bytes of words and the workspaces of small-M calls, masked attention, its
 * gradients, tree attention over 16 and 4 bits and the gradient of norms, if any ran on it.
 * Waits for the stream first (queued kernels may still use them).  For callers
 * that create and destroy streams: call it before destroying a stream the
 * library was used on, from no other thread launching on that stream at the same
 * time.  A later call on the stream allocates afresh.  GSR_OK if the pair holds
 * nothing; GSR_ERR_CUDA if the wait or a free failed.
 */
gsr_status gsr_release_stream(struct CUstream_st* stream);

/* Kernel the library would run for these sizes on the current device: 0 = tiled
 * (one CTA per 128-row tile, 128 x 256, 128 x 128 or 128 x 64 tiles, whichever
 * needs fewer waves with a wave of 256-wide tiles counted as 1.45 and one of 64-wide
 * tiles as 0.9 of a wave of 128-wide ones), 1 = small-M (M <= 64 with B of at
 * least 16 MiB, and 65 to 128
 * rows when B holds at least 64 MiB and those one-CTA tiles would keep under two
 * thirds of the SMs busy),
 * 2 = tiled on CTA pairs with 256 x 256 tiles (for more than 128 rows and K above
 * 384, where a tile is more than its epilogue, chosen when
 * there is at least one full wave of such tiles, or when K >= 6144 and 0 would use
 * 128 x 256 tiles: the pair's faster K loop then repays its larger cost per launch;
 * at 128 rows or fewer a pair tile would be at least half empty), 3 = tiled on CTA
 * pairs with 256 x 128 tiles (instead
 * of 2 where a wave of them, counted as 0.68 of a wide wave, finishes the work at
 * least 5 % sooner: in practice N of about 128, where a 256-wide tile is half
 * empty).  The constants come from measured sweeps on GB300. */
int gsr_select_path(int64_t M, int64_t N, int64_t K);

/* Forces a path for later calls (process-wide): 0 = automatic (default),
 * 1 = tiled with automatic tile width, 2 = small-M (only honoured when
 * M <= 256: 65 to 256 rows run with an MMA N of 128 or 256, which the automatic
 * choice takes only for the 65-128-row case above; the host-buffer entry point's
 * blocks ignore it),
 * 3 = tiled with 128 x 256 tiles, 4 = tiled with 128 x 128 tiles,
 * 5 = tiled on CTA pairs with 256 x 256 tiles, 6 = tiled on CTA pairs with
 * 256 x 128 tiles, 7 = tiled with 128 x 64 tiles.
 * For tests and measurements. */
void gsr_set_path_override(int path);

/* Raster grouping of the tiled kernels (process-wide): `group` consecutive tile rows
 * (M blocks) share each tile column before moving on, so that concurrently running
 * CTAs reuse the same A and B panels from L2 -- the "L2 swizzle" knob of the aikraft.ru
 * TileLang tutorial survey's "Knobs" section (3).  0 restores the default, 16 row
 * blocks per group (128-row blocks for one CTA per tile, 256-row blocks for CTA pairs).
 * The small-M kernel walks K slabs, not a raster, and ignores it.  For tuning and
 * measurements. */
void gsr_set_raster_group(int group);

/* Split-K of the small-M kernel (process-wide): each 128-column tile's K is cut
 * into `slabs` slabs of whole 64-wide k-blocks (at most one slab per k-block), run
 * as separate work items and summed in slab order (deterministic for a given
 * `slabs`).  0 restores the default, as many slabs as fill the SMs once.  The
 * split-K knob of the aikraft.ru TileLang tutorial survey's "Knobs" section (3);
 * for tuning and measurements.  gemm_scale_relu_noalloc ignores it (its fixed
 * scratch is sized for the default split). */
void gsr_set_split_k(int slabs);

/* Upper bound, in nanoseconds, on every wait inside the kernels (default 1 s).
 * A wait that runs out records an error (see gsr_device_status) and the kernel
 * exits early, leaving C incomplete. */
void gsr_set_wait_timeout_ns(uint64_t ns);

/* Test-only switches, 0 in normal use.  Bit 0: the first CTA's producer skips
 * its first shared-memory fill, so that CTA's waits run out (exercises the
 * bounded-wait path without faulting the GPU).  Bit 1: the tiled kernels copy B
 * as separate 64-column boxes even where one 3-D copy per stage would do.
 * Bits 2-7 switch off or swap what the CTA-pair and attention kernels normally
 * do, for measurements: bit 2 every wave of pair tiles walks K forward (no
 * serpentine order); bit 3 C stores without the L2 evict-first hint; bit 4 the
 * first pair's second CTA skips its first fill (like bit 0, on the other CTA);
 * bit 5 / bit 6 B copies with an L2 evict-first / evict-normal hint instead of
 * evict-last; bit 7 causal attention launches one head's query blocks at a time. */
void gsr_set_test_flags(uint32_t flags);

/* CUDA error code of the last failing CUDA call on this host thread (0: none). */
int gsr_last_cuda_error(void);

/* Static, human-readable name of a status. */
const char* gsr_status_string(gsr_status s);

/* Library version string, e.g. "gsr 0.1.0 sm_103a". */
const char* gsr_version(void);

/* Frees every workspace and error word the library holds, on every device.
 * Must not run while work queued by the library is still executing. */
gsr_status gsr_shutdown(void);

#ifdef __cplusplus
}
#endif

#endif /* GSR_H_ */
