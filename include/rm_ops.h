/*
 * rm_ops.h -- one C entry point per step of the scoring hot path.
 *
 * The launchers that rm_score (rm.h) chains are exported here, so that each
 * step can be checked on its own against the fp64 oracle; beside them stand
 * steps that rm_score never takes (the vote, the attention without an
 * allocation, the steps of incremental scoring).  All pointers
 * are DEVICE pointers unless marked host; all work is asynchronous on stream
 * (a cudaStream_t as void*).  Return RM_OK or a negative RM_E_* code (rm.h);
 * arguments are validated on the host before anything is enqueued.
 *
 * Packed varlen layout shared by the steps (TurboTransformers review,
 * "variable-length input" in the abstract; no padding to a fixed length):
 *   offsets[n+1]  int32 token offsets, sequence i = rows offsets[i]..offsets[i+1]-1,
 *                 L_i = offsets[i+1]-offsets[i] >= 1.
 *   X[T][H]       activations, row-major.
 *   QKV[T][3H]    Q in columns 0..H-1, K in H..2H-1, V in 2H..3H-1; head j
 *                 uses columns j*d .. j*d+d-1 of each.
 *   S             attention scores/probabilities.  With Lp_i = round_up(L_i, 8)
 *                 the entry (sequence i, head j, query r, key c) is at
 *                 S[s_off[i] + (j*L_i + r)*Lp_i + c], s_off[i] = sum_{k<i} h*L_k*Lp_k.
 *                 Only c < L_i (causal: c <= r) is ever read or written.
 *   rb_off[n+1]   prefix sums of ceil(L_i/64): the 64-query row blocks that
 *                 the attention launches distribute over CTAs.
 * dtype arguments: RM_F32 (0) or RM_BF16 (1) from rm.h.
 */
#ifndef RM_OPS_H_
#define RM_OPS_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Failure detection of the calls below, which have no handle: waits for the
 * current device, writes how many pipeline waits gave up in the kernels that
 * rm_op_* calls of this process launched there since the last call (0 in normal
 * operation; a kernel that gave one up returned early and its outputs are
 * invalid), and clears the count.  out: host int64.  RM_E_INVAL for NULL,
 * RM_E_CUDA on a CUDA error. */
int rm_op_timeouts(int64_t* out);
/* Failure detection without a fault, as rm_selftest_bounded_wait (rm.h): one
 * thread waits on a barrier that nothing completes, through the wait of
 * rm_op_attn_window, and gives up after limit_ns (1e3 .. 1e10), which the next
 * rm_op_timeouts reports.  Synchronous; the CUDA context stays usable. */
int rm_selftest_op_wait(int64_t limit_ns);

/* Host helper: rb_off[n+1] and s_off[n+1] for the layout above (host arrays).
 * Returns RM_OK, RM_E_INVAL for a length < 1 or non-monotone offsets. */
int rm_varlen_meta(const int32_t* offsets, int32_t n, int32_t n_heads,
                   int32_t* rb_off, int64_t* s_off);

/* Y[M][N] = act(X[M][K] . W[N][K]^T + bias[N]) -- the QKV, output and FFN
 * projections (the "BLAS routines" of the TurboTransformers abstract; tensor
 * cores per its proposed-method section).  bf16 operands, fp32 accumulation
 * in tensor memory (tcgen05), bias/GELU in the epilogue.
 *   x: bf16 [M][K] row-major; w: bf16 [N][K] row-major (nn.Linear layout);
 *   bias: fp32 [N] or NULL; y: [M][N] row-major of y_dtype (RM_F32|RM_BF16).
 *   act: 0 = none, 1 = GELU (erf), 2 = GELU (tanh).
 * Requires M >= 1, N and K multiples of 8, 16-byte aligned x, w, y. */
int rm_op_gemm(const void* x, const void* w, const float* bias, void* y, int32_t y_dtype,
               int32_t M, int32_t N, int32_t K, int32_t act, void* stream);

/* rm_op_gemm with an explicit output tile (the projections of rm_op_gemm; the
 * tile choice itself has no counterpart in the pages and is exposed for
 * testing every tile and for tuning): cg = 1 (one CTA per 128 x bn tile,
 * bn in {64, 96, 128, 160, 192, 224, 256}) or cg = 2 (a cluster of two CTAs
 * per 256 x bn tile on the pair MMA, bn in {128, 192, 256}); cg = 0 takes the
 * tile rm_gemm_tile picks (what rm_op_gemm does).  Same arguments and
 * requirements as rm_op_gemm; RM_E_INVAL for a tile outside these sets. */
int rm_op_gemm_tiled(const void* x, const void* w, const float* bias, void* y, int32_t y_dtype,
                     int32_t M, int32_t N, int32_t K, int32_t act, int32_t cg, int32_t bn,
                     void* stream);

/* Y[M][N] += X[M][K] . W[N][K]^T + bias[N] with Y in fp32: the pre-LN
 * decoder's output projection and FFN2 added straight into its fp32 residual
 * stream (the residual additions of the layer equations, which the
 * TurboTransformers abstract pairs with the LayerNorm batch reduction; here
 * folded into the GEMM that produces the addend).  The tile is accumulated in
 * fp32 and added to y in L2; each element of y is added to exactly once, with
 * one fp32 rounding, so the result equals a separate fp32 addition of the
 * rm_op_gemm output and does not depend on the order of the tiles.  Same
 * arguments as rm_op_gemm_tiled with y_dtype = RM_F32 and act = 0 (RM_E_INVAL
 * for any other); y must be 16-byte aligned and is read and written. */
int rm_op_gemm_accumulate(const void* x, const void* w, const float* bias, void* y,
                          int32_t y_dtype, int32_t M, int32_t N, int32_t K, int32_t act,
                          int32_t cg, int32_t bn, void* stream);

/* Majority vote of an ensemble of K scorer replicas ("experts"), the SambaNova
 * blog's accuracy section (Figs. 4-5: several TinyBERT instances vote on each
 * input).  scores: device float[K][n], expert k's score of input i at
 * scores[k*n + i].  Expert k answers [score > threshold]; decision[i] = 1 when
 * more than K/2 experts answer 1, 0 when fewer, and on an even split 1 iff the
 * margins sum_k (score - threshold), added in expert order in fp32, are > 0.
 * decision, votes: device int32[n], either may be NULL.  RM_E_INVAL for
 * K < 1, n < 0 or NULL scores.  Asynchronous on stream. */
int rm_op_vote(const float* scores, int32_t K, int32_t n, float threshold, int32_t* decision,
               int32_t* votes, void* stream);

/* Host only (no counterpart in the pages): the output tile the projections
 * without an activation use for an M x N x K product on a device with num_sms
 * SMs (a GELU epilogue may take
 * a single-CTA tile where this returns a pair).  out[0] = cg (1 or 2),
 * out[1] = bn.  RM_E_INVAL for M, N, K or num_sms < 1 or out == NULL. */
int rm_gemm_tile(int32_t M, int32_t N, int32_t K, int32_t num_sms, int32_t* out);

/* X[t] = E_word[clamp(ids[t])] + E_pos[t - offsets[i]] for each token t of
 * sequence i, then (ln_g != NULL) the embedding LayerNorm.  ids out of 0..V-1
 * are clamped and counted with atomicAdd into *err_count (may be NULL).
 * E_word: bf16 [V][H]; E_pos: bf16 [P][H]; ln_g, ln_b: fp32 [H] or NULL;
 * x: [T][H] of x_dtype (RM_BF16, or RM_F32 for the decoder's fp32 residual
 * stream).  Requires every L_i <= P. */
int rm_op_embed(const int32_t* ids, const int32_t* offsets, int32_t n_seqs, int32_t T,
                const void* emb_word, const void* emb_pos, const float* ln_g, const float* ln_b,
                float eps, int32_t V, int32_t P, int32_t H, void* x, int32_t x_dtype,
                int32_t* err_count, void* stream);

/* Attention scores S = (Q K^T)/sqrt(d) per sequence and head, only the valid
 * L_i x L_i block (causal: keys c <= r).  qkv: bf16 [T][3H]; S: bf16.
 * n_row_blocks = rb_off[n] (host value); head_dim even, <= 128. */
int rm_op_attn_scores(const void* qkv, void* S, const int32_t* offsets, const int32_t* rb_off,
                      const int64_t* s_off, int32_t n_seqs, int32_t n_row_blocks,
                      int32_t n_heads, int32_t head_dim, int32_t causal, void* stream);

/* Masked row softmax in place over every row of S: p_c = exp(s_c - max)/sum
 * over keys c < L_i (causal: c <= r) -- the Softmax batch reduction of the
 * TurboTransformers abstract.  fp32 math; s_dtype RM_BF16 or RM_F32.
 * T = offsets[n] and max_len >= every L_i (host values). */
int rm_op_softmax(void* S, int32_t s_dtype, const int32_t* offsets, const int64_t* s_off,
                  int32_t n_seqs, int32_t T, int32_t n_heads, int32_t max_len, int32_t causal,
                  void* stream);

/* The same softmax by row-length class: the rows are first regrouped on the
 * device by the 8-element chunks of their length (<= 1, 2, 4, 8, 16, 32, 64,
 * 96, 128) into scratch, each row recording its sequence, and one persistent
 * kernel then takes each class with lanes per row fitted to it (one lane for
 * rows of up to 8 keys ... 32 lanes holding 4 chunks each for 1024), so that
 * short rows leave no lanes idle when the batch also holds long ones and no
 * lane group searches the offsets.  Same arguments as rm_op_softmax, plus
 * scratch: device memory of rm_softmax_scratch_bytes(n_seqs, T, n_heads) bytes
 * (about 4 bytes per row), 16-byte aligned, overwritten by the call.  The
 * per-row arithmetic is rm_op_softmax's; only the order in which a row's
 * exponentials are summed follows its lanes per row.  RM_E_INVAL for NULL
 * pointers or bad sizes. */
int rm_op_softmax_classes(void* S, int32_t s_dtype, const int32_t* offsets, const int64_t* s_off,
                          int32_t n_seqs, int32_t T, int32_t n_heads, int32_t max_len,
                          int32_t causal, void* scratch, void* stream);
/* Host only: the scratch bytes rm_op_softmax_classes needs (0 for bad sizes). */
size_t rm_softmax_scratch_bytes(int32_t n_seqs, int32_t T, int32_t n_heads);

/* Context C = P V per sequence and head into ctx[T][H] (head j in columns
 * j*d..j*d+d-1).  S holds P (bf16), qkv: bf16 [T][3H], ctx: bf16 [T][H]. */
int rm_op_attn_context(const void* S, const void* qkv, void* ctx, const int32_t* offsets,
                       const int32_t* rb_off, const int64_t* s_off, int32_t n_seqs,
                       int32_t n_row_blocks, int32_t n_heads, int32_t head_dim, int32_t causal,
                       void* stream);

/* The three attention steps above in one kernel: per sequence, head and
 * 64-query block, S = QK^T/sqrt(d) over keys c < L_i (causal: c <= r) with an
 * online (running max and sum) softmax, P rounded to bf16, C = P V written to
 * ctx[T][H].  No score buffer.  qkv: bf16 [T][3H]; ctx: bf16 [T][H]. */
int rm_op_attn_fused(const void* qkv, void* ctx, const int32_t* offsets, const int32_t* rb_off,
                     int32_t n_seqs, int32_t n_row_blocks, int32_t n_heads, int32_t head_dim,
                     int32_t causal, void* stream);

/* The same attention step on tiles of 64 consecutive packed rows: a tile
 * holds whole short sequences and pieces of long ones, and each CTA takes one
 * tile and a group of heads, its K/V rows (the tile's key range) arriving by
 * TMA in 64-row chunks while the previous chunk is multiplied.  A query row
 * admits the keys of its own sequence only (c <= r too when causal); online
 * softmax in fp32, P rounded to bf16 for P V, as in rm_op_attn_fused.
 * head_dim 64 or 128 (H = n_heads * head_dim); qkv: bf16 [T][3H]; ctx: bf16
 * [T][H]; offsets: DEVICE int32[n+1] with offsets[n] = T (host value T);
 * max_len: a host bound on every L_i (it sizes the launch: CTAs take fewer
 * heads each when rows are long).  RM_E_INVAL for other head dims or sizes < 1; waits that give up (none in
 * normal operation) are counted (rm_op_timeouts). */
int rm_op_attn_tiles(const void* qkv, void* ctx, const int32_t* offsets, int32_t n_seqs, int32_t T,
                     int32_t n_heads, int32_t head_dim, int32_t max_len, int32_t causal,
                     void* stream);

/* Tiles of the tensor-core attention (rm_op_attn_tc): a greedy cut of the
 * packed batch into runs of whole sequences of at most 128 rows each.
 * offsets: HOST int32[n_seqs+1] with offsets[0] = 0 and every length in
 * 1..128; tiles: HOST int32[n_seqs+1] (caller-owned), receives tiles[0..k]
 * with tiles[0] = 0 and tiles[k] = n_seqs, tile j holding sequences
 * [tiles[j], tiles[j+1]).  Returns k (>= 1), or RM_E_INVAL / RM_E_RANGE.
 * This cut of the batch has no counterpart in the pages; it is the layout
 * of the kernel below. */
int rm_attn_tc_tiles(const int32_t* offsets, int32_t n_seqs, int32_t* tiles);

/* The attention step of rm_op_attn_tiles on the 5th-generation tensor cores,
 * for head_dim 64 and sequences of at most 128 tokens (the TurboTransformers
 * proposed-method section's batched QK^T, batch softmax and PV, fused): per
 * tile of rm_attn_tc_tiles and head, S = QK^T (tcgen05.mma into tensor
 * memory), the row softmax over the row's own sequence (c <= r too when
 * causal) in fp32 with P rounded to bf16, and C = P V (tcgen05.mma), written
 * to ctx.  qkv: bf16 [T][3H], H = 64 * n_heads; ctx: bf16 [T][H]; offsets:
 * DEVICE int32[n_seqs+1] with offsets[n_seqs] = T (host value T); tiles:
 * DEVICE int32[n_tiles+1] as rm_attn_tc_tiles wrote them for the same
 * offsets.  RM_E_INVAL for NULL pointers or sizes < 1; waits that give up
 * (none in normal operation) are counted (rm_op_timeouts). */
int rm_op_attn_tc(const void* qkv, void* ctx, const int32_t* offsets, const int32_t* tiles,
                  int32_t n_tiles, int32_t n_seqs, int32_t T, int32_t n_heads, int32_t causal,
                  void* stream);

/* Work items of the long-row tensor-core attention (rm_op_attn_tcl): every
 * run of 128 query rows of a sequence, item = (sequence << 2) | tile (tile
 * 0..3 covers rows 128*tile ..), those that read the most 128-key chunks
 * first (causal != 0: a tile reads keys up to its own last row only).
 * offsets: HOST int32[n_seqs+1] with offsets[0] = 0 and every length in
 * 1..512; items: HOST int32[4 * n_seqs] (caller-owned).  Returns the item
 * count (sum over sequences of ceil(L / 128)), or RM_E_INVAL / RM_E_RANGE.
 * This cut has no counterpart in the pages; it is the layout of the kernel
 * below. */
int rm_attn_tcl_items(const int32_t* offsets, int32_t n_seqs, int32_t causal, int32_t* items);

/* rm_op_attn_tc for sequences of up to 512 tokens (head_dim 64): per item of
 * rm_attn_tcl_items and head, S = Q K^T for the item's 128 query rows against
 * every 128-key chunk of its sequence (tcgen05.mma into tensor memory), the
 * row softmax over the row's own sequence (c <= r too when causal) in fp32
 * with P rounded to bf16, and C = P V (tcgen05.mma), written to ctx.  qkv:
 * bf16 [T][3H], H = 64 * n_heads; ctx: bf16 [T][H]; offsets: DEVICE
 * int32[n_seqs+1] with offsets[n_seqs] = T (host value T); items: DEVICE
 * int32[n_items] as rm_attn_tcl_items wrote them for the same offsets and
 * causal flag.  RM_E_INVAL for NULL pointers, sizes < 1 or n_items >
 * 4 * n_seqs; waits that give up (none in normal operation) are counted
 * (rm_op_timeouts). */
int rm_op_attn_tcl(const void* qkv, void* ctx, const int32_t* offsets, const int32_t* items,
                   int32_t n_items, int32_t n_seqs, int32_t T, int32_t n_heads, int32_t causal,
                   void* stream);

/* The materialised attention step (rm_op_attn_scores -> rm_op_softmax ->
 * rm_op_attn_context) without any device allocation: the score matrix and the
 * per-call metadata live in one file-scope device array of 8 MiB of scores
 * plus 65,552 bytes of metadata (8,454,160 bytes) that
 * every device loading this library keeps until the process exits.  The pages
 * have no counterpart to this entry point; it exists for callers that cannot
 * allocate device memory where they run the step (a plugin inside another
 * runtime that owns the device memory pool, or a path where cudaMalloc is not
 * allowed because it may synchronize the device or fail under pressure).
 *   qkv: bf16 [T][3H]; ctx: bf16 [T][H] (written); offsets: HOST int32[n+1].
 * Limits: n_seqs <= 4096, every L_i <= 1024 and sum_i n_heads*L_i*round_up(L_i,8)
 * <= 4 Mi score entries; larger calls return RM_E_RANGE (use the three
 * caller-allocated entry points instead).  The first call in a CUDA context (for most
 * callers, the device's primary context) looks up the array's device address
 * (cudaGetSymbolAddress) and caches it for that context; make that first call
 * before any stream capture.  The call copies its metadata into the
 * array on stream and calls no cudaMalloc or cudaFree.  Every call shares the
 * array and it keeps the last call's contents (nothing in it needs to start at
 * zero: each call writes every entry it reads), so calls that overlap on the
 * GPU -- on different streams, or from different threads without ordering --
 * race and give wrong results. */
int rm_op_attention_noalloc(const void* qkv, void* ctx, const int32_t* offsets, int32_t n_seqs,
                            int32_t n_heads, int32_t head_dim, int32_t causal, void* stream);

/* ---------------------------------------------------------------------------
 * Incremental scoring: a text scored as it grows, its keys and values kept in
 * a paged cache instead of being recomputed ("Learning to summarize from human
 * feedback" summary, method section: the reward model is a causal decoder, so
 * earlier tokens' keys and values do not depend on later ones).  A step is
 *   rm_op_kv_slots       where the step's new tokens go in the cache
 *   (QKV projection)     rm_op_gemm
 *   rm_op_qk_norm_rope   per-head norm and rotation of q and k, cache write
 *   rm_op_attn_window    prompts: the new tokens attend to one another, or
 *   rm_op_attn_decode    one new token per sequence attends to the cache.
 * Unlike the steps above, these take grouped heads (n_q_heads a multiple of
 * n_kv_heads; query head j reads key-value head j / (n_q_heads / n_kv_heads))
 * and rows with a pitch (row_stride elements from one token to the next).
 * Every device pointer must belong to the current CUDA device.  One a call
 * (offsets of rm_op_kv_slots, q_out, out) is looked up: host memory or another
 * device's gives RM_E_INVAL; the others are taken on trust.
 * None of them allocates or keeps anything between calls; all can be captured
 * in a CUDA graph.
 * ------------------------------------------------------------------------- */

/* A paged cache.  Element (page p, kv head h, slot s, dim c) of the keys is
 * k[p*page_stride + (h*page_size + s)*head_dim + c]; the values likewise.
 * A token's slot number is p*page_size + s.  dtype RM_BF16, or RM_E4M3: 8-bit
 * floats (4 exponent, 3 mantissa bits) standing for value * scale of the head
 * (k_scale, v_scale: device float[n_kv_heads], > 0; both NULL = 1).  k and v
 * are 16-byte aligned, page_stride (elements) * element size a multiple of 16
 * and page_stride >= n_kv_heads * page_size * head_dim: pages of several
 * layers, or keys beside values, may interleave in one allocation. */
#define RM_E4M3 2
typedef struct rm_kv_cache {
  void* k;
  void* v;
  int64_t page_stride;
  int32_t n_pages;
  int32_t page_size;             /* tokens per page, 1..1024                     */
  int32_t n_kv_heads;
  int32_t head_dim;
  int32_t dtype;                 /* RM_BF16 | RM_E4M3                            */
  const float* k_scale;
  const float* v_scale;
} rm_kv_cache;

/* How positions rotate: pair i of the first rot_dim dims of a head turns by
 * position * freqs[i] radians (freqs: device double[rot_dim/2], see
 * rm_rope_freqs); the other dims stay.  layout RM_ROPE_HALF pairs dims i and
 * i + rot_dim/2, RM_ROPE_INTERLEAVED dims 2i and 2i+1.  The rotated pair is
 * multiplied by mscale (1 for none). */
#define RM_ROPE_HALF        0
#define RM_ROPE_INTERLEAVED 1
typedef struct rm_rope {
  const double* freqs;
  int32_t rot_dim;               /* even, 0..head_dim; 0 = no rotation           */
  int32_t layout;
  float mscale;
} rm_rope;

/* Host only: the turning rates f_i = base^(-2i/rot_dim), i < rot_dim/2, and
 * their changes for contexts longer than a model was trained on:
 *   RM_ROPE_PLAIN    f_i
 *   RM_ROPE_LINEAR   f_i / factor (positions interpolated)
 *   RM_ROPE_BASE     base * factor^(rot_dim/(rot_dim-2)) in place of base, so
 *                    that the slowest pair is stretched by factor and the
 *                    fastest stays (rot_dim > 2)
 *   RM_ROPE_PARTS    per pair, by how often it turns over trained tokens (Peng
 *                    et al., "YaRN: Efficient Context Window Extension of
 *                    Large Language Models", section 3.2): pairs that turn
 *                    more than fast times keep f_i, those that turn less than
 *                    slow times take f_i / factor, between them linearly in
 *                    the number of turns.
 * freqs: host double[rot_dim/2].  factor >= 1; trained >= 1 and fast > slow > 0
 * are read by RM_ROPE_PARTS only.  RM_E_INVAL for anything else. */
#define RM_ROPE_PLAIN  0
#define RM_ROPE_LINEAR 1
#define RM_ROPE_BASE   2
#define RM_ROPE_PARTS  3
int rm_rope_freqs(int32_t rot_dim, double base, int32_t scaling, double factor, double trained,
                  double fast, double slow, double* freqs);

/* Block tables and slot maps of a step, built on the device from the request
 * lengths.  Sequence i holds len_before[i] tokens and gets n_new[i] more (0 or
 * more).  Its tokens need ceil(len / page_size) pages; the ones it lacks come
 * from free_pages[*used_before ..] in request order and are written to its
 * row of block_table ([n_seqs][table_stride]).  Written:
 *   offsets[n_seqs+1]   packed offsets of the new tokens
 *   positions[T], slots[T]  position in the sequence and cache slot of each
 *                       new token; entries behind the last token up to T (a
 *                       padded batch) get position 0 and slot -1
 *   len_after[n_seqs]   len_before + n_new
 *   used_after[1]       *used_before plus the pages taken
 *   unserved[1]         how many sequences did not fit (0 normally): the
 *                       first whose pages exceed n_free, whose new tokens
 *                       exceed T, whose row exceeds table_stride pages or
 *                       whose length is negative, and every one behind it.
 *                       These get no tokens and no pages, and len_after =
 *                       len_before; a later call may serve them.
 * len_after may be len_before and used_after may be used_before (a captured
 * step that advances itself); no other buffers may overlap.  Page numbers of
 * free_pages and of block_table are copied, not checked.  n_seqs <= 16384. */
int rm_op_kv_slots(const int32_t* len_before, const int32_t* n_new, int32_t n_seqs,
                   int32_t page_size, const int32_t* free_pages, int32_t n_free,
                   const int32_t* used_before, int32_t* block_table, int32_t table_stride,
                   int32_t T, int32_t* offsets, int32_t* positions, int64_t* slots,
                   int32_t* len_after, int32_t* used_after, int32_t* unserved, void* stream);

/* Norm and rotation of a projection's queries and keys, and the cache write,
 * in one pass.  Row t of qkv holds the token's query heads, then its key
 * heads, then its value heads, head_dim elements each (bf16).  Per head:
 *   y = x / sqrt(mean(x^2) + eps) * gain      (q_gain, k_gain: fp32 [head_dim],
 *                                              4-byte aligned; both NULL =
 *                                              no norm)
 *   z = y with its first rot_dim dims rotated by positions[t] (rope NULL: z = y)
 * in fp32, rounded once.  The squares of a head must add up to less than 2^128;
 * a head of zeros with eps = 0 is NaN.  The angle position * freqs[i] is
 * computed and freed of whole turns in 64 bits: it is off by at most 3 * 2^-53
 * of itself (with freqs[i] <= 1 less than 2^-24 radians up to position 2^27,
 * 7e-7 at 2^31), and then rounded to fp32.
 * Written: q_out (row t's query heads), k_out (its key heads; NULL = not
 * written), and, when cache != NULL, the key and value heads to slots[t] of the
 * cache (bf16, or x * (1 / scale), both in fp32, rounded to the nearest 8-bit
 * value, +-448 at most, NaN kept).  A token whose slot is negative or beyond
 * the cache's last page is not written to the cache.  Two tokens must not share
 * a slot.  q_out and k_out may be the q and k columns of qkv itself (in place);
 * no other overlap.
 * head_dim a multiple of 8, 8..256; qkv, q_out, k_out 16-byte aligned with
 * strides that are multiples of 8 elements.  T >= 0; T = 0 does nothing, and the
 * buffers with an entry a token may be NULL then (those of an empty tensor). */
int rm_op_qk_norm_rope(const void* qkv, int64_t qkv_stride, void* q_out, int64_t q_stride,
                       void* k_out, int64_t k_stride, int32_t T, int32_t n_q_heads,
                       int32_t n_kv_heads, int32_t head_dim, const float* q_gain,
                       const float* k_gain, float eps, const rm_rope* rope,
                       const int32_t* positions, const rm_kv_cache* cache, const int64_t* slots,
                       void* stream);

/* Causal attention of packed sequences with a sliding window and sinks: token
 * t of a sequence sees its key j <= t when j > t - window or j < sinks (window
 * 0: every j <= t).  out = softmax(q k^T / sqrt(head_dim)) v over the seen
 * keys, fp32 softmax, P rounded to bf16 before the product with V (its rows'
 * sums are taken before that rounding).  q, out: [T][n_q_heads*head_dim], k,
 * v: [T][n_kv_heads*head_dim], bf16, each with its row stride; offsets: DEVICE
 * int32[n_seqs+1], offsets[0] = 0, non-decreasing (empty sequences allowed),
 * offsets[n_seqs] <= T (cut to it); rows behind it are not written.  Values
 * and keys that a row does not see do not reach it, infinities and NaN among
 * them; a row whose seen scores are all -infinity is NaN.  Rows that an unseen
 * infinity or NaN would have reached, and rows whose weights rise by more than
 * 2^40 from one stretch of 128 keys to the next, are computed again by a warp
 * each: exact, but at about 0.5 us a key.  Finite values are taken up to
 * |v| * keys = 2^87 (the sums of p v are divided at the end, and p may reach
 * 2^40 before its reference moves).  out overlaps no input.  head_dim 64 or
 * 128; pointers 16-byte aligned, strides multiples of 8 elements;
 * n_q_heads / n_kv_heads <= 128.  T >= 0; T = 0 does nothing, and q, k, v and
 * out may be NULL then.  Waits that give up (none in normal operation) are
 * counted (rm_op_timeouts); the outputs are then invalid. */
int rm_op_attn_window(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                      const void* v, int64_t v_stride, const int32_t* offsets, int32_t n_seqs,
                      int32_t T, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                      int32_t window, int32_t sinks, void* out, int64_t out_stride, void* stream);

/* The same attention for one new token per sequence over the paged cache: row
 * i of q is the query of the last of length[i] tokens of sequence i, whose
 * keys and values lie in pages block_table[i*table_stride ..] in order (the
 * new token's own among them).  length[i] <= 0 gives a row of zeros; lengths
 * beyond table_stride * page_size are cut to it.  A page number outside
 * 0..n_pages-1 drops its page's tokens.  The work is split over the lengths
 * and joined in a fixed order (the same call gives the same bits); partial
 * results go to workspace: device memory of rm_attn_decode_workspace bytes,
 * 16-byte aligned, overwritten, which no other call may use at the same time
 * (calls captured in graphs that may overlap need workspaces of their own).
 * Pages that a window hides are not read.  P is rounded to bf16 before the
 * product with V as in rm_op_attn_window; over an e4m3 cache it is held in
 * fp16, where weights down to 2^-32 of the largest that the same split of the
 * row holds keep that precision and those below 2^-40 of it reach the sum
 * only.  Queries over an e4m3 cache are held in fp16 too, relative to the
 * largest of their head (entries below 2^-27 of it lose bits).  Finite values are taken up to
 * |v| * keys = 2^127 (the sums of p v are divided at the end).  out overlaps no
 * input.  cache->head_dim 64 or 128. */
int rm_op_attn_decode(const void* q, int64_t q_stride, const rm_kv_cache* cache,
                      const int32_t* block_table, int32_t table_stride, const int32_t* length,
                      int32_t n_seqs, int32_t n_q_heads, int32_t window, int32_t sinks, void* out,
                      int64_t out_stride, void* workspace, size_t workspace_bytes, void* stream);
/* Host only: the workspace bytes of rm_op_attn_decode for up to n_seqs
 * sequences, whatever their lengths (0 for bad sizes). */
size_t rm_attn_decode_workspace(int32_t n_seqs, int32_t n_q_heads, const rm_kv_cache* cache);

/* Residual + LayerNorm over rows of length H (the LayerNorm batch reduction of
 * the TurboTransformers abstract), fp32 math:
 *   mode 0 (post-LN): x = LN(y + x)              (z unused, may be NULL)
 *   mode 1 (pre-LN):  x = y + x;  z = LN(x)      (both written)
 *   mode 2 (plain):   z = LN(x)                  (y unused, may be NULL)
 * LN(u) = g * (u - mean)/sqrt(var + eps) + b with the biased variance.
 * y, x, z: [T][H]; g, b: fp32 [H].  Row types by dtype: RM_F32 or RM_BF16 for
 * all three; RM_ROWS_RESID_F32 for x in fp32 with y and z in bf16;
 * RM_ROWS_F32_IN for y and x in fp32 with z in bf16 (the pre-LN decoder's
 * layout: its residual stream and the sublayer outputs added to it stay fp32,
 * so that each addition is rounded once to fp32 instead of to bf16). */
#define RM_ROWS_RESID_F32 2
#define RM_ROWS_F32_IN 3
int rm_op_res_ln(const void* y, void* x, void* z, const float* g, const float* b, int32_t T,
                 int32_t H, float eps, int32_t dtype, int32_t mode, void* stream);

/* Scalar head ("Learning to summarize from human feedback" summary, method
 * section): out[i] = w_r . u_i + b_r where u_i = x[offsets[i]] (last_token =
 * 0) or x[offsets[i+1]-1] (last_token = 1).  x: bf16 [T][H]; w_r: fp32 [H];
 * out: fp32 [n]. */
int rm_op_head(const void* x, const int32_t* offsets, int32_t n_seqs, const float* w_r,
               float b_r, int32_t H, int32_t last_token, float* out, void* stream);

/* Host only: the arena plan for one call of a handle created with cfg.
 * Fills, for each intermediate buffer k < returned count (<= max_bufs):
 * out_off[k], out_bytes[k] (byte offset/size in the arena), out_first[k],
 * out_last[k] (first and last step that uses it; buffers whose step ranges
 * overlap are live together and never share bytes).  *out_peak = arena bytes
 * the plan needs.  T tokens, n_seqs sequences, s_elems score elements
 * (s_off[n]).  Returns the buffer count or a negative RM_E_* code. */
int rm_arena_plan(const void* cfg, int32_t T, int32_t n_seqs, int64_t s_elems,
                  int64_t* out_off, int64_t* out_bytes, int32_t* out_first, int32_t* out_last,
                  int32_t max_bufs, int64_t* out_peak);

#ifdef __cplusplus
}
#endif
#endif /* RM_OPS_H_ */
