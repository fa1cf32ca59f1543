/*
 * speckv.h -- C ABI of the B200 (sm_100a) lookahead importance-scoring library.
 *
 * The method is "Draft-based Approximate Inference for LLMs" (paper notes,
 * ICLR 2026, arXiv 2506.08373):
 *   - section 关键设计, SpecKV: for every attention head, the queries of the
 *     last n_window input tokens and of the n_lookahead draft (lookahead)
 *     tokens attend to the input keys; the attention that the remaining input
 *     keys receive estimates the importance of each KV pair; the top-C_max KV
 *     pairs plus the window are kept.
 *   - section 关键设计, SpecPC: draft attention A[layer][head][query][key] over
 *     a large query window with weights that fall with distance from the end,
 *     the first l_skip layers skipped, averaged first, then maximised.
 *   - section 关键设计, SpecKV-PC: SpecPC first, then SpecKV on what it kept.
 *   - section 损失函数 / 训练策略: SpecPC smooths scores with local pooling.
 *
 * Conventions for every entry point
 *   - Tensor arguments are DEVICE pointers owned by the caller, contiguous in
 *     the layouts given below, 16-byte aligned.  The library allocates no
 *     memory: scratch space is the caller's `workspace`, whose size comes from
 *     the matching *_workspace_size() query.
 *   - bf16 means IEEE bfloat16 bit patterns (uint16_t); fp32 is float.
 *   - All work is enqueued on `stream` (a cudaStream_t, passed as void*;
 *     NULL = legacy default stream) and returns without host synchronisation.
 *   - The return value is a spk_status.  Argument errors are detected on the
 *     host and returned BEFORE anything is launched; spk_last_error() then
 *     describes the problem (thread-local string).
 *   - Errors found on the device (a bounded wait that timed out, an index
 *     outside its range in kv_compact) are recorded in device error words
 *     that spk_device_error() reads; kernels never trap.
 *   - Results are deterministic: the same inputs give bitwise identical
 *     outputs (no floating-point atomics).
 *   - Calls on the same stream are ordered; calls that share a workspace must
 *     not run concurrently on different streams.
 */
#ifndef SPECKV_H
#define SPECKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SPK_OK = 0,
  SPK_ERR_ARG = 1,          /* a null/misaligned pointer or an inconsistent shape */
  SPK_ERR_UNSUPPORTED = 2,  /* a valid shape outside what the kernels implement */
  SPK_ERR_WORKSPACE = 3,    /* workspace missing or smaller than *_workspace_size() */
  SPK_ERR_CUDA = 4,         /* a CUDA runtime/driver call failed (see spk_last_error) */
  SPK_ERR_TIMEOUT = 5       /* reported by spk_device_error: a device wait ran out */
} spk_status;

/* ------------------------------------------------------------------------
 * SpecKV scoring (section 关键设计, SpecKV)
 *
 * A unit is one (batch element, layer, KV head); units are numbered
 * u = (b * layers + l) * hkv + h.  Query head qh belongs to KV head qh / g,
 * g = hq / hkv (GQA).  R = n_window + n_lookahead query rows per query head:
 * row i < n_window is the window query at input position n_in - n_window + i
 * and sees input keys 0 .. n_in - n_window + i (causal); row i >= n_window is
 * a lookahead (draft) query and sees all n_in input keys.  Keys of the
 * lookahead tokens are not input keys and are not part of the softmax.
 *
 *   q      bf16 [batch][layers][hq][R][head_dim]   (rows pre-scaled or not: see scale)
 *   k      bf16 [batch][layers][hkv][n_in][head_dim]
 *   scores fp32 [units][n_pre], n_pre = n_in - n_window:
 *          scores[u][j] = sum over the g query heads of unit u and their R rows
 *                         of softmax_j(scale * q_row . k_j)   (prefix keys only)
 *   window_mass fp32 [units][n_window] or NULL: the same sum on the window keys
 *          j = n_pre .. n_in-1 (every prefix and window column together sum to
 *          g * R per unit, which makes it a conservation check).
 *
 * Supported: head_dim in {64, 128}; hq % hkv == 0; g * R <= 2048;
 * 0 <= n_window <= n_in; R >= 1; scale > 0 and finite.
 * ------------------------------------------------------------------------ */
typedef struct {
  int batch, layers, hq, hkv, head_dim;
  int n_in, n_window, n_lookahead;
  float scale; /* multiplies q.k before the softmax (1.0 if q is pre-scaled) */
} spk_speckv_shape;

/* Workspace: the row offsets pass 1 hands to pass 2, 32 bytes per query row
 * with each unit's g * R rows rounded up to 128:
 * units * ceil(g * R / 128) * 4096 bytes (rounded up to 256); 16-byte aligned. */
size_t speckv_workspace_size(const spk_speckv_shape* shape);

spk_status speckv_score(const spk_speckv_shape* shape, const void* q_bf16, const void* k_bf16,
                        float* scores, float* window_mass, void* workspace, size_t workspace_bytes,
                        void* stream);

/* The two passes of speckv_score as separate calls, for callers that time
 * or schedule them apart; speckv_score is exactly speckv_row_offsets
 * followed by speckv_colsum on the same stream.
 *   speckv_row_offsets: pass 1 -- every query row's log-sum-exp, stored in the
 *     workspace as the row offsets pass 2 adds to its logits;
 *   speckv_colsum: pass 2 -- the scores (and window mass) from a workspace that
 *     speckv_row_offsets filled for the same shape, q and k (ordered before
 *     this call; the workspace is only read).
 * Same shapes, layouts, workspace size and rules as speckv_score. */
spk_status speckv_row_offsets(const spk_speckv_shape* shape, const void* q_bf16, const void* k_bf16,
                              void* workspace, size_t workspace_bytes, void* stream);

spk_status speckv_colsum(const spk_speckv_shape* shape, const void* q_bf16, const void* k_bf16, float* scores,
                         float* window_mass, const void* workspace, size_t workspace_bytes, void* stream);

/* Pass 1 alone (diagnostic): the log2-domain log-sum-exp of every query row,
 * lse2[u][qh_local * R + i] = log2 sum_{visible j} 2^(scale*log2(e) * q.k_j),
 * fp32 [units][g * R].  Same shapes and rules as speckv_score. */
spk_status speckv_row_lse(const spk_speckv_shape* shape, const void* q_bf16, const void* k_bf16,
                          float* lse2, void* stream);

/* speckv_score for callers that cannot allocate device memory.  The paper
 * has no counterpart: this is a deployment variant.  Serving engines that
 * reserve nearly all of HBM for their own KV-cache pool, and plugin hosts
 * that give plugins no access to the CUDA allocator, can neither cudaMalloc
 * nor spare a workspace; this call keeps pass 1's row offsets in a fixed
 * 16 MiB array inside the library image instead (no allocation of any kind).
 *   - Same shapes, layouts, outputs and rules as speckv_score.
 *   - Rejects (SPK_ERR_UNSUPPORTED, before any launch) shapes whose workspace
 *     (speckv_workspace_size) would exceed 16 MiB, i.e. more than 524,288
 *     query rows with each unit's rows rounded up to 128.
 *   - Every GPU that loads the library holds the 16 MiB until process exit.
 *   - The first call on a device looks up the array's address on that device
 *     (cudaGetSymbolAddress) and caches it: make it before any stream capture.
 *     A cudaDeviceReset unloads the library's device image, so the cached
 *     address is stale afterwards: do not call this entry point again in a
 *     process that has reset the device.
 *   - All calls share the array, which keeps the last call's contents (every
 *     entry read is first rewritten by the same call, so nothing needs
 *     clearing); calls whose kernels overlap on the GPU race on it. */
spk_status speckv_score_static_ws(const spk_speckv_shape* shape, const void* q_bf16, const void* k_bf16,
                                  float* scores, float* window_mass, void* stream);

/* ------------------------------------------------------------------------
 * Prefill attention of the window and lookahead rows (section 关键设计,
 * SpecKV: the input tokens and the lookahead tokens go through the target
 * model's prefill together, and the importance scores are read from the
 * attention of the last n_window input rows and of the lookahead rows)
 *
 * The key/value sequence of a unit is its n_in input tokens followed by its
 * n_lookahead lookahead tokens.  Query row i of a head (R = n_window +
 * n_lookahead rows, ordered as for speckv_score) sits at position
 * n_in - n_window + i and attends causally to the keys up to that position:
 *   out[u][row]   = softmax_j(scale * q_row . k_j) . v_j over those keys
 *   lse2[u][row]  = log2 sum_{j < min(pos + 1, n_in)} 2^(scale*log2(e) * q_row . k_j)
 *                   -- the same input-key normaliser as speckv_row_lse
 *   workspace     = (when non-NULL) the row offsets exactly as
 *                   speckv_row_offsets writes them, so that speckv_colsum on
 *                   the same shape, q and k gives the importance scores
 *                   without the scoring's own first pass.
 *
 *   q              bf16 [batch][layers][hq][R][head_dim]
 *   k, v           bf16 [batch][layers][hkv][n_in][head_dim]         (input tokens)
 *   k_look, v_look bf16 [batch][layers][hkv][n_lookahead][head_dim]  (NULL if n_lookahead = 0)
 *   out            bf16 [batch][layers][hq][R][head_dim]
 *   lse2           fp32 [units][g * R] or NULL
 *   workspace      NULL, or speckv_workspace_size(shape) bytes, 16-byte aligned
 * Probabilities enter the P.V product as bf16 (fp32 accumulation); the
 * normaliser and lse2 are formed from the fp32 probabilities.
 * Supported: as speckv_score.
 * ------------------------------------------------------------------------ */
spk_status speckv_prefill_attention(const spk_speckv_shape* shape, const void* q_bf16, const void* k_bf16,
                                   const void* v_bf16, const void* k_look_bf16, const void* v_look_bf16,
                                   void* out_bf16, float* lse2, void* workspace, size_t workspace_bytes,
                                   void* stream);

/* ------------------------------------------------------------------------
 * Vertical-Slash sparse prefill attention (section 损失函数 / 训练策略: SpecKV
 * runs the target prefill with Vertical-Slash sparse attention, the pattern
 * of the cited sparse-attention work)
 *
 * Per unit (batch element, layer, KV head) the pattern is a set of vertical
 * key columns and a set of slash diagonals (offsets o = p - j).  The query
 * row at position p attends to the keys j <= p with j in vertical, or
 * p - j in slash, or j = p (a token always sees itself):
 *   out[u*g + h][i] = softmax_j(scale * q . k_j) . v_j over those keys,
 *   lse2[u*g + h][i] = log2 sum_j 2^(scale*log2(e) * q . k_j)   (optional)
 * Query rows are the last n_q positions: row i sits at n - n_q + i.
 *
 *   q         bf16 [batch][layers][hq][n_q][head_dim]
 *   k, v      bf16 [batch][layers][hkv][n][head_dim]
 *   vertical  int32 [units][n_vertical], ascending, unique, in [0, n)
 *   slash     int32 [units][n_slash], ascending, unique, in [0, n)
 *   out       bf16 [batch][layers][hq][n_q][head_dim]
 *   lse2      fp32 [units * g][n_q] or NULL
 *   workspace vs_workspace_size(shape) bytes (the vertical keys' K and V rows,
 *             gathered on the stream first), 16-byte aligned; may be NULL when
 *             n_vertical = 0
 * A vertical or slash entry outside [0, n) is ignored and recorded as
 * SPK_ERR_ARG in the device error word; unsorted lists give wrong results.
 * Probabilities enter the P.V product as bf16 (fp32 accumulation).
 * Supported: head_dim in {64, 128}; hq % hkv == 0; 1 <= n_q <= n <= 65536;
 * n_vertical <= 4096; n_slash <= n.
 * ------------------------------------------------------------------------ */
typedef struct {
  int batch, layers, hq, hkv, head_dim;
  int n, n_q, n_vertical, n_slash;
  float scale;
} spk_vs_shape;

size_t vs_workspace_size(const spk_vs_shape* shape);

spk_status vs_sparse_attention(const spk_vs_shape* shape, const void* q_bf16, const void* k_bf16,
                               const void* v_bf16, const int32_t* vertical, const int32_t* slash, void* out_bf16,
                               float* lse2, void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * SpecPC scoring (section 关键设计, SpecPC)
 *
 * Per batch element b, the draft's last W = n_rows query positions: row i sits
 * at position n_in + n_lookahead - 1 - W + i and sees input keys 0 .. that
 * position (capped at n_in - 1).  For every query head qh and layer
 * l >= l_skip, P[l][qh][i][j] is the causal softmax of scale * q . k_j.
 *   S[qh][j] = ( sum_{l >= l_skip} sum_i w_i P[l][qh][i][j] ) / ( sum_i w_i * (layers - l_skip) )
 *   scores[b][j] = max_qh S[qh][j]        for j in 0 .. n_in-1
 *
 *   q            bf16 [batch][layers][hq][W][head_dim]   (layers < l_skip are not read)
 *   k            bf16 [batch][layers][hkv][n_in][head_dim]
 *   row_weights  fp32 [W], device, oldest row first, w_i >= 0, sum > 0; a row
 *                of weight 0 contributes nothing (its attention is not read)
 *   scores       fp32 [batch][n_in]
 *
 * Supported: head_dim in {64, 128}; hq % hkv == 0; hq <= 32; (hq/hkv) * W <= 2048;
 * 0 <= l_skip < layers; 1 <= W <= n_in + n_lookahead - 1; n_lookahead >= 1.
 * ------------------------------------------------------------------------ */
typedef struct {
  int batch, layers, l_skip, hq, hkv, head_dim;
  int n_in, n_rows, n_lookahead;
  float scale;
} spk_specpc_shape;

/* Workspace: the row offsets, units * ceil((hq/hkv) * W / 128) * 4096 bytes
 * (rounded up to 256), units = batch * (layers - l_skip) * hkv; when the
 * column pass would leave SMs of the current device idle (few 256-key blocks,
 * e.g. batch 1 at 32K), it splits each block's (KV head, layer) segments into
 * G groups (G <= 16, chosen from the device's SM count) and adds
 * batch * ceil(n_in / 256) * G * hq * 1 KB of per-head partial sums, which a
 * merge kernel adds in a fixed order (results stay bitwise reproducible on a
 * given device).  Query the size with the device current; 16-byte aligned. */
size_t specpc_workspace_size(const spk_specpc_shape* shape);

spk_status specpc_score(const spk_specpc_shape* shape, const void* q_bf16, const void* k_bf16,
                        const float* row_weights, float* scores, void* workspace, size_t workspace_bytes,
                        void* stream);

/* The two passes of specpc_score as separate calls (specpc_score is exactly
 * specpc_row_offsets followed by specpc_colsum on the same stream): the row
 * offsets with the row weights folded in, then the scores from them. */
spk_status specpc_row_offsets(const spk_specpc_shape* shape, const void* q_bf16, const void* k_bf16,
                              const float* row_weights, void* workspace, size_t workspace_bytes, void* stream);

spk_status specpc_colsum(const spk_specpc_shape* shape, const void* q_bf16, const void* k_bf16, float* scores,
                         void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Pooling + top-k selection (section 关键设计: keep the top-C_max KV pairs plus
 * the window; section 损失函数 / 训练策略: local pooling keeps token runs)
 *
 * For each of `units` rows of n_cand candidate scores, r = pool_kernel / 2 and
 * W_j = [j - r, j + r] ∩ [0, n_cand) (the window clipped at the row's ends):
 *   pooled[j] = max of scores over W_j                 (SPK_POOL_MAX)
 *             = (sum of scores over W_j) / |W_j|       (SPK_POOL_AVG; fp32, summed
 *               in index order, one correctly rounded division)
 *   selected  = the min(k, n_cand) largest pooled values; equal values are
 *               taken lowest index first
 *   idx[u]    = selected indices in ascending order, then the tail
 *               n_cand, n_cand + 1, .., n_cand + n_tail - 1 (the kept window)
 *
 *   scores  fp32 [units][n_cand], finite (NaN order is unspecified; -0 == +0)
 *   idx     int32 [units][min(k, n_cand) + n_tail]
 *   pooled  fp32 [units][n_cand] or NULL
 *
 * The pages say "local pooling" without its kind; the workloads use max
 * pooling, which is what topk_select does.  topk_select_pool takes the mode.
 * Workspace: units * round_up(n_cand, 4) * 4 bytes, 16-byte aligned (the
 * order-preserving 32-bit keys of the pooled values, one padded row per
 * unit).  It is required by the contract; rows of up to 327,680 candidates
 * with pool_kernel <= 2049 keep their keys in shared memory instead and
 * leave it untouched.
 *
 * Supported: pool_kernel odd >= 1; k >= 0; n_tail >= 0; n_cand >= 0;
 * pool_mode SPK_POOL_MAX or SPK_POOL_AVG.
 * ------------------------------------------------------------------------ */
typedef enum {
  SPK_POOL_MAX = 0,
  SPK_POOL_AVG = 1
} spk_pool_mode;

size_t topk_workspace_size(int units, int n_cand);

spk_status topk_select(const float* scores, int units, int n_cand, int pool_kernel, int k, int n_tail,
                       int32_t* idx, float* pooled, void* workspace, size_t workspace_bytes, void* stream);

spk_status topk_select_pool(const float* scores, int units, int n_cand, int pool_mode, int pool_kernel, int k,
                            int n_tail, int32_t* idx, float* pooled, void* workspace, size_t workspace_bytes,
                            void* stream);

/* ------------------------------------------------------------------------
 * KV compaction (section 关键设计, SpecKV: the dropped cache keeps only the
 * selected KV pairs)
 *
 *   k_out[u][t] = k[u][ idx[u / units_per_idx][t] ],  same for v
 *   k, v         [units][n_src][head_dim] elements of elem_bytes bytes
 *   idx          int32 [units / units_per_idx][n_idx], each in [0, n_src)
 *   k_out, v_out [units][n_idx][head_dim]
 * units_per_idx = 1 gives every unit its own index row; units_per_idx =
 * layers * hkv shares one row across all (layer, KV head) of a batch element
 * (SpecPC / SpecKV-PC).  v and v_out may both be NULL.  Rows are copied
 * byte for byte.  An index outside [0, n_src) leaves that output row
 * unwritten and records SPK_ERR_ARG in the device error word.  k and v may
 * be device addresses of pinned host memory (spk_mapped_host_pointer): only
 * the selected rows are then read over the host link.
 *
 * Supported: head_dim * elem_bytes a multiple of 16; units % units_per_idx == 0.
 * ------------------------------------------------------------------------ */
spk_status kv_compact(const void* k, const void* v, int units, int n_src, int head_dim, int elem_bytes,
                      const int32_t* idx, int n_idx, int units_per_idx, void* k_out, void* v_out,
                      void* stream);

/* ------------------------------------------------------------------------
 * Decode attention over a compacted cache (section 整体框架: the target model
 * then runs on the compressed KV cache; section 关键设计, SpecKV: the cache
 * holds the kept KV pairs).  One new query token per attention head:
 *
 *   out[b][l][qh][:] = sum_t softmax_t(scale * q[b][l][qh] . k[b][l][qh/g][t]) * v[b][l][qh/g][t]
 *   q      bf16 [batch][layers][hq][head_dim]
 *   k, v   bf16 [batch][layers][hkv][n_kv][head_dim]   (e.g. kv_compact's outputs)
 *   out    fp32 [batch][layers][hq][head_dim]
 * The softmax runs over all n_kv rows (the caller appends the new token's own
 * K/V row when it should attend to itself).  Deterministic.
 *
 * Supported: head_dim in {64, 128}; hq % hkv == 0; hq / hkv <= 8; n_kv >= 1;
 * scale > 0 and finite.
 * ------------------------------------------------------------------------ */
spk_status decode_attention(int batch, int layers, int hq, int hkv, int head_dim, int n_kv, float scale,
                            const void* q_bf16, const void* k_bf16, const void* v_bf16, float* out,
                            void* stream);

/* ------------------------------------------------------------------------
 * A paged KV cache (section 整体框架: the target model goes on decoding over
 * the reduced cache; the paper does not say how the cache is kept)
 *
 *   k_pages, v_pages [layers][n_pages][hkv][page_rows][head_dim], elements of
 *                    elem_bytes bytes; a page holds page_rows rows of every
 *                    layer and KV head
 *   page_table       int32 [n_seqs][max_pages]: row t of sequence s is row
 *                    t % page_rows of page page_table[s][t / page_rows]; -1
 *                    where the sequence has no page
 *   seq_lens         int32 [n_seqs]: the rows of each sequence
 *   page_refs        int32 [n_pages]: how many sequences hold the page (0: free)
 * An empty cache has page_table = -1, seq_lens = 0 and page_refs = 0.  All of
 * it is on the device and is changed there, in stream order.  Sequences may
 * hold pages together (kv_pages_fork); rows are only ever written into pages
 * that one sequence holds.
 *
 * Lists of sequences (seqs, src, dst) are int32 device arrays of n <= 1024
 * entries.  *result (int32, device) tells what became of a call: 0 done; > 0
 * that many free pages were missing; -1 an argument was wrong (a sequence, its
 * length or a count out of range, a destination listed twice), recorded as SPK_ERR_ARG in
 * the device error word too.  Unless it is 0 the call changed nothing.  Free
 * pages are taken lowest number first, for the sequences in the list's order.
 * page_table, seq_lens, page_refs and the lists need 4-byte alignment, the
 * pages 16.
 * Calls that change the same cache must not overlap on different streams.
 *
 * Supported: head_dim * elem_bytes a multiple of 16; max_pages * page_rows,
 * n * max_pages, layers * n_pages * hkv < 2^31.
 * ------------------------------------------------------------------------ */
typedef struct {
  int layers, n_pages, hkv, page_rows, head_dim, elem_bytes;
  int n_seqs, max_pages;
} spk_pages_shape;

/* Workspace of kv_pages_reserve, kv_pages_compact and kv_pages_fork over n
 * sequences: 4 * (n * max_pages + 4 n) bytes (rounded up to 256); 16-byte
 * aligned. */
size_t kv_pages_workspace_size(const spk_pages_shape* shape, int n);

/* Sequence seqs[i] grows by n_new[i] >= 0 rows: seq_lens, and pages for the
 * rows that have none (the rows themselves are left to kv_pages_write).  A
 * partially filled last page that other sequences hold too is replaced by a
 * copy of its rows, unless n_new[i] is 0.  No sequence may be listed twice. */
spk_status kv_pages_reserve(const spk_pages_shape* shape, void* k_pages, void* v_pages, int32_t* page_refs,
                            int32_t* page_table, int32_t* seq_lens, const int32_t* seqs, const int32_t* n_new, int n,
                            int32_t* result, void* workspace, size_t workspace_bytes, void* stream);

/* The newest rows of each sequence: for unit u = (i * layers + l) * hkv + h and
 * t < counts[i],
 *   row seq_lens[seqs[i]] - counts[i] + t of sequence seqs[i] = k[u][idx[u / units_per_idx][t]],  same for v
 *   k, v    [n][layers][hkv][n_src][head_dim]
 *   idx     int32 [n * layers * hkv / units_per_idx][n_idx], each in [0, n_src);
 *           NULL: row t is row t of k (n_idx <= n_src)
 *   counts  int32 [n], each in [0, n_idx]; NULL: n_idx
 * e.g. a prompt's rows (idx NULL), the rows topk_select kept (units_per_idx 1),
 * or the accepted nodes of a token tree (units_per_idx layers * hkv).  reserved
 * (int32, device) is the *result of the kv_pages_reserve that made room for the
 * rows: nothing is written unless it is 0; NULL: there was room.  A row whose index or position is out of range, or whose page is held by another
 * sequence too, is left unwritten and recorded as SPK_ERR_ARG in the device
 * error word; so are the rows of an entry whose sequence stands earlier in the list. */
spk_status kv_pages_write(const spk_pages_shape* shape, const void* k, const void* v, int n_src, const int32_t* idx,
                          int n_idx, int units_per_idx, const int32_t* counts, const int32_t* page_refs,
                          const int32_t* page_table, const int32_t* seq_lens, const int32_t* seqs, int n,
                          void* k_pages, void* v_pages, const int32_t* reserved, void* stream);

/* Sequence dst[i] becomes the n_idx rows of sequence src[i] that idx selects,
 * in pages of its own (kv_compact for a paged cache):
 *   row t of dst[i] = row idx[u / units_per_idx][t] of src[i], for u = (i * layers + l) * hkv + h
 *   idx  int32 [n * layers * hkv / units_per_idx][n_idx], each in [0, seq_lens[src[i]])
 * What dst[i] held is released; src[i] keeps its rows unless it is a
 * destination of the call (dst[i] == src[i] compacts in place).  The sources
 * are read as they were before the call; no destination may be listed twice.
 * An index out of range leaves that row unwritten and is recorded as
 * SPK_ERR_ARG in the device error word. */
spk_status kv_pages_compact(const spk_pages_shape* shape, void* k_pages, void* v_pages, int32_t* page_refs,
                            int32_t* page_table, int32_t* seq_lens, const int32_t* src, const int32_t* dst, int n,
                            const int32_t* idx, int n_idx, int units_per_idx, int32_t* result, void* workspace,
                            size_t workspace_bytes, void* stream);

/* Sequence dst[i] becomes the rows of sequence src[i] as it was before the call
 * (its first n_rows[i] rows where n_rows is given and that is fewer), by
 * holding their pages: no row is copied.  What dst[i] held is released.  No
 * destination may be listed twice; a source may, and may be a destination (a
 * beam search's reordering).  Of the shape, head_dim, elem_bytes, layers and
 * hkv are not used. */
spk_status kv_pages_fork(const spk_pages_shape* shape, int32_t* page_refs, int32_t* page_table, int32_t* seq_lens,
                         const int32_t* src, const int32_t* dst, const int32_t* n_rows, int n, int32_t* result,
                         void* workspace, size_t workspace_bytes, void* stream);

/* Sequence seqs[i] keeps its first keep_rows[i] rows (none where keep_rows is
 * NULL); pages behind them are released.  A sequence listed twice keeps the
 * fewer; an entry out of range is skipped and recorded as SPK_ERR_ARG in the
 * device error word.  Of the shape, head_dim, elem_bytes, layers and hkv are
 * not used. */
spk_status kv_pages_free(const spk_pages_shape* shape, int32_t* page_refs, int32_t* page_table, int32_t* seq_lens,
                         const int32_t* seqs, const int32_t* keep_rows, int n, void* stream);

/* ------------------------------------------------------------------------
 * Attention for a tree of drafted tokens over a paged cache (section 整体框架:
 * a draft model runs ahead of the target; here the target checks its tokens
 * together)
 *
 * Batch element b has T = n_nodes drafted tokens (nodes) behind sequence
 * s = seqs[b], of which the first n_live[b] count.  Node i of query head qh
 * attends to the seq_lens[s] rows of the cache and to the nodes j < n_live[b]
 * with bit j % 32 of mask[b][i][j / 32] set:
 *   out[b][l][qh][i]  = softmax(scale * q . k) . v over those keys
 *   lse2[b][l][qh][i] = log2 sum 2^(scale * log2(e) * q . k)   (optional)
 * A node that sees no key, or whose logits are all -inf, gets out = 0 and
 * lse2 = -inf.  Rows of nodes
 * i >= n_live[b] are left as they were.  T = 1 is single-token decoding.
 *
 *   q               [batch][layers][hq][T][head_dim]
 *   k_pages, v_pages [layers][n_pages][hkv][page_rows][head_dim]
 *   page_table      int32 [n_seqs][max_pages], seq_lens int32 [n_seqs]
 *   seqs            int32 [batch] or NULL (element b is sequence b)
 *   k_tree, v_tree  [batch][layers][hkv][T][head_dim]; both NULL: the nodes see
 *                   the cache only
 *   mask            32-bit words [batch][T][ceil(T / 32)] (tree_mask), or NULL:
 *                   node i sees the nodes 0 .. i (a chain)
 *   n_live          int32 [batch] or NULL (T)
 *   out             like q; lse2 fp32 [batch][layers][hq][T] or NULL
 *   workspace       tree_attention_workspace_size(shape) bytes, 16-byte
 *                   aligned, for the shape's device (query it with that device
 *                   current): the partial results of units that several CTAs
 *                   share.  It needs no clearing.
 * q, pages, tree and out are bf16 or fp16 (dtype).  Rows behind a sequence's
 * length or among the nodes that do not count are never read into a result,
 * whatever they hold.  What is not finite in the V of a node that a row sees
 * adds to that row however small its weight (inf stays inf, inf - inf is NaN);
 * in the V of a cached row it leaves the column inf, -inf or NaN.  An element
 * whose sequence, length or node count is out of range keeps its output rows and
 * is recorded as SPK_ERR_ARG in the device error word; a page number out of range
 * is recorded and its rows are read as zeros.  Weights enter the V product
 * rounded to dtype (fp32 accumulation); the normaliser and lse2 are formed from
 * the fp32 weights.
 * Supported: head_dim in {64, 128}; hq % hkv == 0; T <= 1024; batch <= 1024;
 * page_rows a multiple of 8; layers * n_pages * hkv and the key tiles (of 64)
 * of all units < 2^31; scale > 0 and finite.
 * ------------------------------------------------------------------------ */
typedef enum {
  SPK_BF16 = 0,
  SPK_FP16 = 1
} spk_dtype;

typedef struct {
  int batch, layers, hq, hkv, head_dim, n_nodes;
  int n_pages, page_rows, n_seqs, max_pages;
  int dtype; /* spk_dtype */
  float scale;
} spk_tree_shape;

size_t tree_attention_workspace_size(const spk_tree_shape* shape);

spk_status tree_attention(const spk_tree_shape* shape, const void* q, const void* k_pages, const void* v_pages,
                          const int32_t* page_table, const int32_t* seq_lens, const int32_t* seqs,
                          const void* k_tree, const void* v_tree, const uint32_t* mask, const int32_t* n_live,
                          void* out, float* lse2, void* workspace, size_t workspace_bytes, void* stream);

/* The visibility words of trees given by their nodes' parents:
 *   parents int32 [batch][n_nodes]: the node before node i, in [-1, i); -1:
 *           node i follows the cache's last row
 *   mask    words [batch][n_nodes][ceil(n_nodes / 32)]: bit j of node i is set
 *           where j is i or one of its ancestors; 0 for nodes >= n_live[b]
 *   depth   int32 [batch][n_nodes] or NULL: how many ancestors a node has (its
 *           position is seq_lens + depth); 0 for nodes >= n_live[b]
 * A parent outside [-1, i) counts as -1, an n_live outside [0, n_nodes] as the
 * nearer end; both are recorded as SPK_ERR_ARG in the device error word.
 * Supported: n_nodes <= 1024; batch <= 65535. */
spk_status tree_mask(int batch, int n_nodes, const int32_t* parents, const int32_t* n_live, uint32_t* mask,
                     int32_t* depth, void* stream);

/* Device address of page-locked, device-mapped host memory (a deployment
 * helper; the paper has no counterpart).  k and v of kv_compact may point
 * into such memory: the gather then reads only the selected rows over the
 * host link instead of copying the whole cache to the device first.
 *   host  a pointer into memory from cudaHostAlloc / cudaHostRegister (any
 *         offset into the allocation)
 *   *dev  the address kernels use for it (owned by the caller's allocation)
 * Returns SPK_ERR_CUDA (and leaves *dev untouched) when the memory is not
 * page-locked and mapped, or no device is present. */
spk_status spk_mapped_host_pointer(const void* host, void** dev);

/* ------------------------------------------------------------------------
 * Errors
 * ------------------------------------------------------------------------ */
/* Message for the last non-OK status returned on this thread ("" if none). */
const char* spk_last_error(void);

/* Synchronises the current device, then reports an error recorded by a
 * kernel since the last clear: *status = SPK_OK, SPK_ERR_TIMEOUT (a bounded
 * device wait ran out; *site says where) or SPK_ERR_ARG (an index out of
 * range in kv_compact, vs_sparse_attention, the kv_pages operators,
 * tree_attention or tree_mask).  Each source file of the
 * library keeps its own first-error word; the first set one, in a fixed
 * order of the files, is reported.  clear != 0 resets them all.  Returns
 * SPK_ERR_CUDA if the device could not be read. */
spk_status spk_device_error(int* status, int* site, int clear);

/* Diagnostic: y[i] = 2^t[i] as computed on the FMA pipe by the scoring
 * epilogues (range reduction + fitted degree-4 polynomial, relative error
 * <= 2.7e-6 for t in [-126, 64); arguments below -126 give a value under
 * 1.2e-38).  t, y: fp32 device arrays of n elements. */
spk_status spk_exp2_fma(const float* t, float* y, int n, void* stream);

/* Self-test of the bounded waits: launches one kernel that waits on a barrier
 * nothing will complete, with a limit of limit_ns nanoseconds (clamped to
 * [1e3, 1e9]).  The kernel gives up, records SPK_ERR_TIMEOUT at site 999 and
 * returns; read it with spk_device_error().  No GPU state is left behind. */
spk_status spk_selftest_wait_timeout(long long limit_ns, void* stream);

/* Self-test of the waits of tree_attention: the call, and in front of it one
 * more run of its main kernel in which two CTAs lose part of their work, as a
 * copy or a warp that never arrives would.  Their waits run out (2 s), record
 * SPK_ERR_TIMEOUT at a site of 600 and more, and the CTAs end; the call behind
 * it, on the same workspace, gives its results.  bf16, head_dim 64, hq / hkv *
 * n_nodes up to 8 or 33 to 128. */
spk_status spk_selftest_tree_give_up(const spk_tree_shape* shape, const void* q, const void* k_pages, const void* v_pages,
                                     const int32_t* page_table, const int32_t* seq_lens, const int32_t* seqs,
                                     const void* k_tree, const void* v_tree, const uint32_t* mask, const int32_t* n_live,
                                     void* out, float* lse2, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPECKV_H */
