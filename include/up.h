/*
 * up.h -- C ABI of the UniPrefill block-sparsification hot path for GB300 (sm_103a).
 *
 * UniPrefill drops unimportant tokens during long-context prefill.  At one
 * full-attention layer the last n queries of each sequence score fixed blocks
 * of G key tokens; the highest-scoring blocks are kept until their cumulative
 * score reaches p; the hidden states and position ids of the kept tokens are
 * gathered into a compacted batch that every later layer consumes.
 *
 * Sources: "UniPrefill: 블록 단위 동적 희소화를 통한 범용적 롱 컨텍스트 프리필 가속화"
 * (aitrends.kr overview; paragraphs on block-wise importance estimation, top-p
 * selection, system integration and sparsity propagation) and the UniPrefill
 * abstract (chatpaper.ai; continuous-batching operator).
 *
 * Conventions shared by every call
 *   - All pointers are DEVICE pointers unless stated otherwise.  The caller
 *     allocates and owns every buffer, including the workspace.  The library
 *     never allocates, frees or synchronises; every call is asynchronous and
 *     ordered on `stream`.
 *   - Sequences are continuously batched (varlen): `cu_seqlens` is int32
 *     [num_seqs + 1], cu_seqlens[0] = 0, non-decreasing, and
 *     cu_seqlens[num_seqs] = total_tokens.  L_s = cu_seqlens[s+1] - cu_seqlens[s].
 *   - Tensors are token-major, row-major and contiguous unless a call says
 *     otherwise; "bf16" buffers hold IEEE bfloat16 values.
 *   - nb_s = ceil(L_s / G) blocks per sequence; cu_blocks is int32
 *     [num_seqs + 1], the exclusive prefix sum of nb_s.
 *   - Host-checkable arguments are validated before any launch; a rejected
 *     call launches nothing and returns the error.  Errors found on the device
 *     (a malformed cu_seqlens, a sequence beyond a kernel's size limit, a
 *     page index outside the key pool, an expired bounded wait) set a sticky
 *     device error word that
 *     up_get_device_error() reports; the affected outputs are then unspecified.
 *   - Functions are thread-safe; the first call on a device queries its
 *     attributes and sets kernel attributes for it.
 */
#ifndef UP_H_
#define UP_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t; NULL is the legacy default stream. */
typedef struct CUstream_st *up_stream_t;

typedef enum {
    UP_OK = 0,
    UP_ERR_INVALID_ARG = 1,  /* null pointer, bad size, p out of range, misaligned buffer */
    UP_ERR_UNSUPPORTED = 2,  /* valid but outside what the kernels implement (head_dim, G, ...) */
    UP_ERR_WORKSPACE = 3,    /* workspace pointer null or smaller than the *_workspace() size */
    UP_ERR_CUDA = 4,         /* a CUDA runtime/driver call failed (launch, attribute, tensor map) */
    UP_ERR_TIMEOUT = 5,      /* a bounded device-side wait expired (reported by up_get_device_error) */
    UP_ERR_DEVICE = 6        /* a device-side argument check failed (reported by up_get_device_error) */
} up_status;

/* Device error bits reported by up_get_device_error(). */
#define UP_DEVERR_BAD_CU_SEQLENS 0x1u  /* cu_seqlens[0] != 0, decreasing, or last != total_tokens */
#define UP_DEVERR_SELECT_TOO_MANY_BLOCKS 0x2u /* a sequence has more than UP_SELECT_MAX_BLOCKS blocks */
#define UP_DEVERR_TIMEOUT 0x4u         /* a bounded wait inside a kernel gave up */
#define UP_DEVERR_BAD_PAGE 0x8u        /* a page index outside [0, num_pages) (read as zeros) */
#define UP_DEVERR_BAD_CU_BLOCKS 0x10u  /* compaction: cu_blocks[num_seqs] < 0 or > total_tokens/G + num_seqs */
#define UP_DEVERR_BOUNDS 0x20u         /* checked builds only (compiled with -DUP_CHECK_BOUNDS; the scoring,
                                          selection and compaction kernels): an index
                                          range outside its buffer; the access was skipped */
#define UP_DEVERR_BAD_KV_LENS 0x40u    /* kv_lens[s] negative, below the sequence's new tokens, or above
                                          max_pages * page_size (the sequence is left out) */

#define UP_DEVERR_BAD_TREE 0x80u       /* drafted tokens: a parent that does not come before its child, or more
                                          than UP_TREE_MAX tokens (the sequence's rows are those of an empty
                                          mask); a fork from a sequence that is none (the child is empty) */
#define UP_DEVERR_NO_PAGES 0x100u      /* the pool has too few free pages for the call */
#define UP_DEVERR_BAD_REFS 0x200u      /* a page released that nobody holds, or pool counts that cannot be */

/* Largest nb_s that the selection calls rank on chip (1M tokens at G = 64). */
#define UP_SELECT_MAX_BLOCKS 16384

/* Static text for a status code. */
const char *up_status_string(up_status status);

/*
 * Block scoring.
 *
 * Source: UniPrefill overview, block-wise importance estimation paragraph (the
 * last n queries are dotted with all keys; block scores come from softmax
 * attention mass) and drop-criterion paragraph (tokens whose softmax
 * probability is near zero are dropped).
 *
 * For sequence s let n_s = min(n, L_s).  Query t in [0, n_s) sits at absolute
 * position a_t = L_s - n_s + t and sees keys i <= a_t (causal).  For query head
 * h (KV head j = h / (Hq/Hk)):
 *     P[h,t,i] = softmax_i( q[t,h,:] . k[i,j,:] / sqrt(d) )   over i <= a_t
 *     scores[cu_blocks[s] + b] = (1 / (n_s*Hq)) * sum_{h,t} sum_{i in block b} P[h,t,i]
 * so each sequence's scores sum to 1.  Block b covers tokens [bG, min((b+1)G, L_s)).
 *
 *   q_last     bf16 [sum_s n_s, Hq, d]: the last n_s query rows of every
 *              sequence, packed in sequence order (RoPE already applied).
 *   k          bf16 [total_tokens, Hk, d] keys (RoPE already applied).
 *   cu_seqlens int32 [num_seqs+1].
 *   Hq, Hk     query / KV heads, Hq % Hk == 0, Hq/Hk <= 16.
 *   d          head_dim: 64, 128 or 256.
 *   n          observation window (last queries), 1 <= n <= 1024.
 *   G          block size: 16, 32, 64, 128 or 256.
 *   scores     fp32 [sum_s nb_s] (output).  Capacity needed: at most
 *              total_tokens/G + num_seqs entries.
 *   cu_blocks  int32 [num_seqs+1] (output).
 *   workspace  device scratch of at least up_score_blocks_workspace(...) bytes,
 *              256-byte aligned; its contents on entry do not matter.
 * Scores are deterministic: a repeat call on the same inputs returns the same bits.
 */
size_t up_score_blocks_workspace(int num_seqs, int64_t total_tokens, int Hq, int Hk, int d,
                                 int n, int G);

up_status up_score_blocks(const void *q_last, const void *k, const int32_t *cu_seqlens,
                          int num_seqs, int64_t total_tokens, int Hq, int Hk, int d, int n,
                          int G, float *scores, int32_t *cu_blocks, void *workspace,
                          size_t workspace_bytes, up_stream_t stream);

/*
 * Block scores of one tensor-parallel shard of the heads.
 *
 * Source: UniPrefill overview, fused-kernel paragraph: under tensor
 * parallelism each rank scores the heads it holds and the block scores are
 * summed across ranks (an all-reduce) before the selection.
 *
 * Exactly up_score_blocks for the Hq query / Hk KV heads this rank holds
 * (q_last [sum n_s, Hq, d], k [total_tokens, Hk, d], whole GQA groups), except
 * that the mean over heads divides by Hq_total, the query heads of all ranks:
 * score_b = sum over this shard's rows of the block's softmax mass, divided by
 * n_s * Hq_total.  The sum of these scores over a partition of all heads into
 * shards is the up_score_blocks score of all heads (up to fp32 rounding); each
 * shard's scores sum to Hq / Hq_total per sequence.  Hq_total == Hq gives
 * up_score_blocks bit for bit.  Same workspace (up_score_blocks_workspace with
 * this shard's Hq, Hk), outputs and errors as up_score_blocks, plus
 * UP_ERR_INVALID_ARG for Hq_total < Hq.
 */
up_status up_score_blocks_shard(const void *q_last, const void *k, const int32_t *cu_seqlens,
                                int num_seqs, int64_t total_tokens, int Hq, int Hk, int d, int n,
                                int G, int Hq_total, float *scores, int32_t *cu_blocks,
                                void *workspace, size_t workspace_bytes, up_stream_t stream);

/*
 * Block scores with the keys in a paged KV cache (chunked prefill).
 *
 * Sources: Chunked Prefill glossary, how-chunking-works section (a long prompt
 * is prefilled in chunks and each chunk attends to the cached keys of the
 * earlier ones); CompactAttention review, key-terms section (paged attention
 * over a KV-head-major cache).
 *
 * Exactly up_score_blocks, except where the keys are read: key t of sequence s
 * (0 <= t < L_s) is row t % page_size of KV head j in page
 * block_table[s * max_pages + t / page_size] of
 *   k_pages   bf16 [num_pages, Hk, page_size, d]  (KV-head-major pages).
 * The query rows of a chunk are its last n_s tokens, as for up_score_blocks,
 * and a sequence's keys are all of its cached tokens, earlier chunks first.
 *   block_table  int32 [num_seqs * max_pages]; entries past a sequence's pages
 *                are not read.
 *   page_size    a multiple of 128 (a 128-key step never straddles two pages).
 * Errors: as up_score_blocks; UP_ERR_INVALID_ARG for a null table, page_size
 * not a positive multiple of 128, num_pages < 1, num_pages * Hk * page_size
 * >= 2^31, or max_pages < 1; a sequence with more than max_pages * page_size
 * tokens sets UP_DEVERR_BAD_CU_SEQLENS (nothing is scored); a page index
 * outside [0, num_pages) sets UP_DEVERR_BAD_PAGE and its keys read as zeros.
 * The workspace is up_score_blocks_workspace's.
 */
up_status up_score_blocks_paged(const void *q_last, const void *k_pages, int64_t num_pages,
                                int page_size, const int32_t *block_table, int max_pages,
                                const int32_t *cu_seqlens, int num_seqs, int64_t total_tokens,
                                int Hq, int Hk, int d, int n, int G, float *scores,
                                int32_t *cu_blocks, void *workspace, size_t workspace_bytes,
                                up_stream_t stream);

/*
 * The kept blocks as a block-CSR matrix (sequences x key blocks) for a
 * block-sparse attention consumer.
 *
 * Source: FlashPrefill V2 review, key-terms section (the active blocks are
 * handed to the sparse-attention kernel as a CSR index).
 *
 *   keep, cu_blocks  as produced by up_select_topp / up_select_blocks and
 *                    up_score_blocks (cu_blocks int32 [num_seqs+1]).
 *   indptr   int32 [num_seqs+1] (output): indptr[s] = kept blocks of the
 *            sequences before s; indptr[num_seqs] = all kept blocks.
 *   indices  int32 [sum nb_s] (output, capacity): entries indptr[s] ..
 *            indptr[s+1]-1 are the kept block numbers of sequence s (0-based
 *            within the sequence), ascending.
 * One CTA; no workspace.  Errors: UP_ERR_INVALID_ARG for a null pointer or
 * num_seqs < 0.
 */
up_status up_block_csr(const uint8_t *keep, const int32_t *cu_blocks, int num_seqs,
                       int32_t *indptr, int32_t *indices, up_stream_t stream);

/*
 * Top-p block selection.
 *
 * Source: UniPrefill overview, top-p selection paragraph: blocks sorted by
 * score are kept until their cumulative sum reaches p (e.g. 0.99).
 *
 * Per sequence, blocks are ranked by (score descending, block index
 * ascending); the cumulative score is taken exactly in rank order (each fp32
 * score as a 64-bit fixed-point multiple of 2^-62, truncated); the kept set is
 * the shortest prefix whose cumulative score is >= p, crossing block included
 * (block at rank r kept iff the mass ranked before it is < ceil(p * 2^62)).
 * p >= 1 keeps every block; if rounding leaves the total below p, every block
 * is kept.
 *
 *   scores, cu_blocks  as produced by up_score_blocks: block masses >= 0 that
 *                      sum to about 1 per sequence (a score >= 1 counts as 1;
 *                      a total above 2 gives an unspecified kept set).
 *   cu_seqlens         int32 [num_seqs+1] (block lengths for kept_tokens).
 *   p                  0 < p; p >= 1 keeps all.
 *   keep               uint8 [sum nb_s] (output): 1 kept, 0 dropped, original order.
 *   kept_tokens        int32 [num_seqs] (output): tokens in the kept blocks.
 * Sequences with nb_s > UP_SELECT_MAX_BLOCKS raise UP_DEVERR_SELECT_TOO_MANY_BLOCKS.
 */
up_status up_select_topp(const float *scores, const int32_t *cu_blocks,
                         const int32_t *cu_seqlens, int num_seqs, int G, double p,
                         uint8_t *keep, int32_t *kept_tokens, up_stream_t stream);

/* Selection rule of up_select_blocks. */
typedef enum { UP_SELECT_TOP_P = 0, UP_SELECT_TOP_K = 1 } up_select_mode;

/* up_select_blocks flag: also keep the last block of every non-empty sequence. */
#define UP_SELECT_KEEP_LAST 0x1u

/*
 * Block selection, general form.
 *
 * Sources: UniPrefill overview, top-p selection paragraph (top-p),
 * hyper-parameters paragraph (its ablation sets top-p against keeping a fixed
 * number of blocks: top-k), system-integration paragraph (decode continues
 * from the end of each sequence: the keep-last option).
 *
 * Blocks are ranked per sequence exactly as in up_select_topp (score
 * descending, block index ascending).
 *   mode UP_SELECT_TOP_P  the kept set of up_select_topp with threshold p
 *                         (0 < p; k is ignored).
 *   mode UP_SELECT_TOP_K  the first min(k, nb_s) ranks (k >= 1; p is ignored).
 *   flags                 0, or UP_SELECT_KEEP_LAST: after the rule, the last
 *                         block of every non-empty sequence is kept too and
 *                         counted in kept_tokens (the method as the pages state
 *                         it leaves this off).
 * The other arguments, outputs and device errors are those of up_select_topp;
 * an unknown mode or flag bit, p <= 0 or NaN in top-p mode, or k < 1 in top-k
 * mode return UP_ERR_INVALID_ARG before any launch.
 */
up_status up_select_blocks(const float *scores, const int32_t *cu_blocks,
                           const int32_t *cu_seqlens, int num_seqs, int G, up_select_mode mode,
                           double p, int k, uint32_t flags, uint8_t *keep, int32_t *kept_tokens,
                           up_stream_t stream);

/*
 * Compaction (sparsity propagation).
 *
 * Source: UniPrefill overview, sparsity-propagation paragraph (every later
 * sub-layer takes only the kept tokens) and system-integration paragraph (the
 * positions of dropped/kept tokens travel with the batch so decode addresses
 * the right KV-cache slots).
 *
 * For each sequence in order and each kept block in ascending order, the
 * block's rows of x and pos are appended to x_out / pos_out.  Positions are
 * gathered, not renumbered.
 *
 *   x               bf16 [total_tokens, hidden], 16-byte aligned; hidden % 8 == 0.
 *   pos             int32 [total_tokens].
 *                   x and pos may be device memory, or pinned (page-locked) host
 *                   memory that the device addresses through unified addressing
 *                   (cudaHostAlloc, cudaHostRegister): the kernel then reads only
 *                   the kept rows across the host link, in place.
 *   keep, cu_blocks as produced above.
 *   x_out           bf16 [capacity, hidden], 16-byte aligned; capacity must be
 *                   >= the number of kept tokens (total_tokens is always enough).
 *   pos_out         int32 [capacity].
 *   cu_seqlens_out  int32 [num_seqs+1] (output): cu_seqlens of the compacted batch.
 *   src_idx         int32 [capacity] or NULL: source row of every output row.
 *   total_kept      int32 [1] (output): number of kept rows (= cu_seqlens_out[num_seqs]).
 *   workspace       at least up_compact_workspace(...) bytes, 256-byte aligned.
 * The output size lives on the device; reading it on the host is the caller's
 * choice (one device-to-host copy of total_kept).  A cu_blocks that cannot be
 * this batch's (its last entry negative or above total_tokens/G + num_seqs;
 * for one sequence, anything but {0, ceil(total_tokens/G)}) sets
 * UP_DEVERR_BAD_CU_BLOCKS and total_kept is 0; nothing is read or written out
 * of bounds, and the other outputs are unspecified.
 */
size_t up_compact_workspace(int num_seqs, int64_t total_tokens, int G);

up_status up_compact(const void *x, const int32_t *pos, int hidden, const int32_t *cu_seqlens,
                     int num_seqs, int64_t total_tokens, int G, const uint8_t *keep,
                     const int32_t *cu_blocks, void *x_out, int32_t *pos_out,
                     int32_t *cu_seqlens_out, int32_t *src_idx, int32_t *total_kept,
                     void *workspace, size_t workspace_bytes, up_stream_t stream);

/*
 * Compaction without a caller-supplied workspace.
 *
 * The UniPrefill pages have no counterpart of this entry point; it exists for
 * callers that cannot allocate device memory when they compact -- an engine
 * that has reserved nearly all HBM for its KV cache, or a serving loop that
 * must not call cudaMalloc because it can synchronise the device.
 *
 * It computes exactly what up_compact computes, with the same arguments minus
 * the workspace.  Its scratch (kept-block list, per-block destination rows and
 * a counter, about 1.3 MB) is a fixed array inside the library that every GPU
 * loading the library holds until the process exits; the call itself
 * allocates and frees nothing.
 *   - Limit: total_tokens / G + num_seqs <= UP_COMPACT_NOALLOC_MAX_BLOCKS
 *     (4M tokens at G = 64); larger batches return UP_ERR_WORKSPACE and launch
 *     nothing.
 *   - The first call on each device looks up the array's device address
 *     (cudaGetSymbolAddress) with that device current; make that first call
 *     before any stream capture.
 *   - All calls on a device share the one array.  Each call rewrites every
 *     scratch entry it reads, so no clearing is needed, but calls that overlap
 *     on the GPU (different streams, no ordering between them) race on it and
 *     give wrong results.
 */
#define UP_COMPACT_NOALLOC_MAX_BLOCKS 65536

up_status up_compact_noalloc(const void *x, const int32_t *pos, int hidden,
                             const int32_t *cu_seqlens, int num_seqs, int64_t total_tokens, int G,
                             const uint8_t *keep, const int32_t *cu_blocks, void *x_out,
                             int32_t *pos_out, int32_t *cu_seqlens_out, int32_t *src_idx,
                             int32_t *total_kept, up_stream_t stream);

/*
 * Paged KV cache: the cache that up_score_blocks_paged reads its keys from, with
 * the values and (optionally) the token positions beside them.
 *
 * Slot i of sequence s (0 <= i < kv_lens[s]) is row i % page_size of page
 * block_table[s * max_pages + i / page_size].
 *   k_pages, v_pages  dtype [num_pages, Hk, page_size, d], 16-byte aligned.
 *   pos_pages    int32 [num_pages, page_size], 16-byte aligned, or NULL: the position
 *                of the token in each slot (a compacted batch's slots are denser than its
 *                positions).  up_append_kv writes it; a distance bias reads it.
 *   block_table  int32 [num_seqs * max_pages]; entries past a sequence's pages
 *                are not read.  A page index outside [0, num_pages) sets
 *                UP_DEVERR_BAD_PAGE: nothing is written there, and its keys,
 *                values and positions read as zeros.
 *   kv_lens      int32 [num_seqs]: cached tokens of each sequence, the tokens of
 *                the current call included.  A length outside [new tokens,
 *                max_pages * page_size], or of 2^31 - 2^16 and more, sets UP_DEVERR_BAD_KV_LENS: the sequence
 *                is not appended to, and its attention output rows are those of
 *                an empty mask.
 *   page_size    a positive multiple of 16 (128 where up_score_blocks_paged reads
 *                the pages too).
 *   d            64, 128 or 256.
 *   dtype        UP_BF16 or UP_FP16 (queries and outputs have the same type).
 * The struct is read on the host during the call; the caller keeps it.
 */
typedef enum { UP_BF16 = 0, UP_FP16 = 1 } up_dtype;

typedef struct {
    void *k_pages;
    void *v_pages;
    int32_t *pos_pages;
    const int32_t *block_table;
    const int32_t *kv_lens;
    int64_t num_pages;
    int32_t num_seqs;
    int32_t max_pages;
    int32_t page_size;
    int32_t Hk;
    int32_t d;
    int32_t dtype; /* up_dtype */
} up_paged_kv;

/*
 * Append: rotates the new tokens' queries and keys by their positions and writes
 * keys, values and positions to the cache, in one kernel.
 *
 * Token t of sequence s (cu_seqlens[s] <= t < cu_seqlens[s+1]) goes to slot
 * kv_lens[s] - (cu_seqlens[s+1] - t).  Frequency i < rot_dim/2 turns its pair of
 * dims by the angle pos[axes[i] * total_tokens + t] * inv_freq[i]:
 *     (a, b) -> (a cos - b sin, b cos + a sin)
 * where (a, b) are dims (i, i + rot_dim/2), or (2i, 2i+1) with
 * UP_ROPE_INTERLEAVED; dims from rot_dim on are copied.  The angle is reduced in
 * 2^-64 turns before its sine and cosine; the frequency in turns is rounded once, to
 * 2^-56 for up to 1 radian a position, so the farthest position's angle is off by 2^-25
 * turns.
 *
 *   q, k, v    dtype [total_tokens, Hq | Hk | Hk, d] with token strides q_stride,
 *              k_stride, v_stride in elements (views of a fused projection are
 *              fine); heads are adjacent.  16-byte aligned, strides multiples of
 *              8 and at least the heads' elements.  Hq = 0 with q = q_out = NULL
 *              appends only.
 *   pos        int32 [num_axes, total_tokens]; pos_pages receives axis 0.
 *   axes       int32 [rot_dim/2] in [0, num_axes), or NULL (all 0); an entry
 *              outside counts as axis 0.
 *   inv_freq   fp32 [rot_dim/2], radians per position; NULL when rot_dim = 0.
 *   rot_dim    0, or a multiple of 16 up to d.
 *   q_out      dtype [total_tokens, Hq, d] contiguous; may be q itself when
 *              q_stride = Hq * d.
 * The tokens' pages must not be shared between sequences.  Where cu_seqlens is
 * malformed (UP_DEVERR_BAD_CU_SEQLENS), a token that lies in no range of it, or in one that
 * ends past total_tokens, is rotated but not appended.  Errors:
 * UP_ERR_INVALID_ARG for null pointers, sizes, strides or alignments outside the
 * above; UP_ERR_UNSUPPORTED for a d or dtype outside the cache's list.
 */
#define UP_ROPE_INTERLEAVED 0x1u

up_status up_append_kv(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                       const void *v, int64_t v_stride, const int32_t *pos, int num_axes,
                       const int32_t *axes, const float *inv_freq, int rot_dim, uint32_t flags,
                       const int32_t *cu_seqlens, int64_t total_tokens, int Hq,
                       const up_paged_kv *cache, void *q_out, up_stream_t stream);

/*
 * How attention turns a query-key product into a logit, and what a query sees.
 *   scale     logits are scale * (q . k) ...
 *   softcap   ... then softcap * tanh(logit / softcap) when softcap > 0 (1e-6 and
 *             more) ...
 *   slopes    fp32 [Hq] or NULL: ... then minus slopes[h] * |q_pos - pos_pages|
 *             (needs q_pos and the cache's pos_pages; a sequence's positions lie within
 *             2^31 - 1 of one another) ...
 *   q_pos     int32 [queries] or NULL.
 * Softmax is over the visible slots only; a query that sees none gives zeros and
 * a log-sum of -infinity.  What is stored in slots that no query of the call sees has
 * no effect, infinities and NaN included, and pages without a visible slot need no
 * valid entry in the block table.
 */
typedef struct {
    float scale;
    float softcap;
    const float *slopes;
    const int32_t *q_pos;
} up_logits;

/*
 * Attention of new tokens over the paged cache (chunked prefill; the cache
 * already holds the new tokens' own keys and values).
 *
 *   q        dtype [total_tokens, Hq, d], the new tokens of every sequence, packed
 *            by cu_seqlens (int32 [num_seqs+1]); Hq % Hk == 0, Hq/Hk <= 16; query
 *            head h reads KV head h / (Hq/Hk).
 *   visible  int32 [total_tokens, 2] (8-byte aligned) or NULL: query t sees slots visible[t][0] <= i
 *            < visible[t][1], cut to [0, kv_lens[s]): windows, packed documents and
 *            bidirectional prefixes are such ranges.  NULL: causal, slots up to the
 *            token's own.
 *   out      dtype [total_tokens, Hq, d]; may not overlap q.
 *   lse      fp32 [total_tokens, Hq] or NULL: natural log of the softmax's sum.
 *   workspace  up_attend_paged_workspace(...) bytes, 256-byte aligned; its contents
 *            on entry do not matter.
 * A malformed cu_seqlens (UP_DEVERR_BAD_CU_SEQLENS) gives every token the output of an
 * empty mask.
 * A cached value that some query of the call may not see but another one may
 * has to be finite (its zero weight multiplies it).  Results are deterministic on
 * a given GPU model (the parts' boundaries depend on its number of SMs).  Each weight of the
 * softmax is rounded once to the cache's type before it multiplies a value; up_decode_attend keeps what
 * that rounding leaves.  So a token's row here and the same token's row there differ by
 * roundings of the type, which matters to whoever compares them bit by bit or breaks near ties.
 * Errors: as above; UP_ERR_INVALID_ARG for slopes without q_pos or pos_pages, a
 * softcap below 0 or between 0 and 1e-6, or a non-finite scale or softcap.
 */
size_t up_attend_paged_workspace(int64_t total_tokens, int num_seqs, int Hq, int Hk, int d);

up_status up_attend_paged(const void *q, const int32_t *cu_seqlens, int64_t total_tokens, int Hq,
                          const up_paged_kv *cache, const up_logits *logits,
                          const int32_t *visible, void *out, float *lse, void *workspace,
                          size_t workspace_bytes, up_stream_t stream);

/*
 * Attention of one new token per sequence over the paged cache (decode): every
 * sequence's length is split over the GPU and the parts are joined.
 *
 *   q         dtype [num_seqs, Hq, d].
 *   kv_start  int32 [num_seqs] or NULL: the first visible slot (a sliding window);
 *             the query sees slots max(kv_start[s], 0) .. kv_lens[s] - 1.
 *             A length of 0 (an idle row of the batch) is fine and sees none.
 *   out, lse  as in up_attend_paged, [num_seqs, Hq, d] and [num_seqs, Hq].
 *   workspace up_decode_attend_workspace(...) bytes, 256-byte aligned; its contents
 *             on entry do not matter.
 * What is stored in a slot that the query does not see has no effect.
 */
size_t up_decode_attend_workspace(int num_seqs, int Hq, int Hk, int d);

up_status up_decode_attend(const void *q, int Hq, const up_paged_kv *cache,
                           const up_logits *logits, const int32_t *kv_start, void *out,
                           float *lse, void *workspace, size_t workspace_bytes,
                           up_stream_t stream);

/*
 * Attention with first tokens that stay visible: up_attend_paged and
 * up_decode_attend where a query sees, beside its window, the first `sinks` slots of
 * its sequence -- as many of them as lie before the window's end.
 *
 * Query t sees slot i iff i < end and (i >= first or i < sinks), with first and end from
 * visible[t] (cut to [0, kv_lens[s])), or kv_start[s] and kv_lens[s].  The pages between
 * the first slots and the window are not read and need no valid entry in the block table.
 *   sinks    0 .. UP_SINKS_MAX (0: the calls above; so is a NULL visible or kv_start, which
 *            leaves nothing between the two).
 * Everything else, the workspaces too, is as for those calls.  UP_ERR_INVALID_ARG for
 * sinks below 0, UP_ERR_UNSUPPORTED above UP_SINKS_MAX.
 */
#define UP_SINKS_MAX 4096

up_status up_attend_sinks(const void *q, const int32_t *cu_seqlens, int64_t total_tokens, int Hq,
                          const up_paged_kv *cache, const up_logits *logits,
                          const int32_t *visible, int sinks, void *out, float *lse,
                          void *workspace, size_t workspace_bytes, up_stream_t stream);

up_status up_decode_sinks(const void *q, int Hq, const up_paged_kv *cache,
                          const up_logits *logits, const int32_t *kv_start, int sinks, void *out,
                          float *lse, void *workspace, size_t workspace_bytes,
                          up_stream_t stream);

/*
 * Attention of a tree of drafted tokens over the paged cache (speculative decoding: the
 * cache already holds the drafted tokens' own keys and values, one slot each, in the order of
 * the call).
 *
 * The n_s = cu_seqlens[s+1] - cu_seqlens[s] drafted tokens of sequence s are its last n_s
 * cached ones.  Each sees the slots before them, from kv_start on and the first
 * `sinks`, and of the drafted ones itself, its parent, its parent's parent and so on.
 *
 *   q         dtype [total_tokens, Hq, d], packed by cu_seqlens, as in up_attend_paged.
 *   parents   int32 [total_tokens]: the parent's number among the sequence's drafted tokens, less
 *             than the token's own, or -1 for one that follows the cache.  A sequence with any
 *             other parent, or of more than UP_TREE_MAX drafted tokens, sets
 *             UP_DEVERR_BAD_TREE and its rows are those of an empty mask.
 *   kv_start  int32 [total_tokens] or NULL: the first slot that each token sees of those
 *             before the drafted ones (a window that moves with a token's depth).  It hides no
 *             ancestor, so a model's window that is shorter than the tree is deep is not
 *             reproduced.
 *   sinks     as in up_attend_sinks.
 *   workspace up_attend_tree_workspace(...) bytes, 256-byte aligned; its contents on entry
 *             do not matter.
 * Values, determinism, the weights' rounding and errors are as in up_attend_paged.
 */
#define UP_TREE_MAX 256

size_t up_attend_tree_workspace(int64_t total_tokens, int num_seqs, int Hq, int Hk, int d);

up_status up_attend_tree(const void *q, const int32_t *cu_seqlens, const int32_t *parents,
                         int64_t total_tokens, int Hq, const up_paged_kv *cache,
                         const up_logits *logits, const int32_t *kv_start, int sinks, void *out,
                         float *lse, void *workspace, size_t workspace_bytes,
                         up_stream_t stream);

/*
 * Compaction of the paged cache in place: of the last n_s = cu_seqlens[s+1] - cu_seqlens[s]
 * cached tokens of every sequence those that are kept move together, in order, right behind
 * the tokens before them -- the accepted path of a drafted tree, or the blocks of a
 * prompt that up_select_blocks kept.  Keys, values and positions move; the slots behind the
 * kept tokens hold what they held.
 *
 *   max_tokens  what cu_seqlens[num_seqs] is at most (above: UP_DEVERR_BAD_CU_SEQLENS); it sizes
 *               the workspace.
 *   keep        uint8 [num_flags]: token i of the n_s is kept iff keep[cu_blocks[s] + i / G].
 *   cu_blocks   int32 [num_seqs+1]: where each sequence's ceil(n_s / G) flags begin (more are
 *               allowed); NULL with G = 1: cu_seqlens.  A sequence whose flags do not fit there,
 *               or reach past num_flags, sets UP_DEVERR_BAD_CU_BLOCKS.
 *   G           tokens of a flag, positive.
 *   kv_lens_out int32 [num_seqs]: the cached tokens that remain, kv_lens[s] - n_s + kept (kv_lens
 *               itself is allowed; other overlaps with it, cu_seqlens or cu_blocks are refused).
 *               Where the caches of several layers share kv_lens, only the last layer's call may
 *               write it: an earlier one would have the others compact the wrong slots, and no
 *               error would tell.
 *   workspace   up_compact_kv_workspace(...) bytes, 256-byte aligned; its contents on entry do
 *               not matter.
 * Pages that hold kept tokens of the n_s, or the slots that they move to, must not be shared between
 * sequences (nor with one that up_fork_pages made).  A sequence with an error (UP_DEVERR_BAD_KV_LENS,
 * UP_DEVERR_BAD_CU_BLOCKS) keeps its cache and length, and so do all under a malformed cu_seqlens
 * (UP_DEVERR_BAD_CU_SEQLENS); a token whose old or new page is outside the pool does not
 * move (UP_DEVERR_BAD_PAGE).  The move's waits are bounded like those of the attention
 * kernels (UP_DEVERR_TIMEOUT: the cache's contents are then unspecified).
 * Errors: as for the calls above; UP_ERR_INVALID_ARG for a cu_blocks of NULL with G > 1.
 */
size_t up_compact_kv_workspace(int64_t max_tokens, int num_seqs, int Hk, int d);

up_status up_compact_kv(const up_paged_kv *cache, const int32_t *cu_seqlens, int64_t max_tokens,
                        const uint8_t *keep, int64_t num_flags, const int32_t *cu_blocks, int G,
                        int32_t *kv_lens_out, void *workspace, size_t workspace_bytes,
                        up_stream_t stream);

/*
 * The pool of a cache's pages, on the device: sequences grow, fork and shrink without the
 * host knowing a length.  One pool serves the caches of all layers that share a block table.
 *   refs        int32 [num_pages]: how many block-table entries hold each page.
 *   free_pages  int32 [num_pages]: a stack; its first num_free entries are the free pages.
 *   num_free    int32 [1].
 * A new pool has no holders, all pages on the stack and block tables of -1.  Calls on one pool
 * (or one block table) are ordered by the caller: one stream, or events.  Tables and stack
 * come out the same in every run.  A num_free outside [0, num_pages] sets UP_DEVERR_BAD_REFS, and the
 * call changes neither pool nor table (a fork's children are all empty).  A stack entry that is no
 * page sets it too, and whoever takes it goes without.
 */
typedef struct {
    int32_t *refs;
    int32_t *free_pages;
    int32_t *num_free;
    int64_t num_pages;
} up_page_pool;

/*
 * Reserve: every entry of row s of block_table that belongs to the tokens have[s] <= t < want[s]
 * -- the entries i with have[s] <= i * page_size < want[s] -- and is negative gets a free
 * page, in the order of (s, i), from the top of the stack down.  Entries that hold a page
 * keep it.  Where the stack ends (UP_DEVERR_NO_PAGES) the entries left stay as they are.  A want
 * above max_pages * page_size sets UP_DEVERR_BAD_KV_LENS and leaves the sequence out.
 *   block_table  int32 [num_seqs, max_pages] (num_seqs * max_pages below 2^31).
 */
up_status up_reserve_pages(const up_page_pool *pool, int32_t *block_table, int num_seqs,
                           int max_pages, int page_size, const int32_t *have, const int32_t *want,
                           up_stream_t stream);

/*
 * Release: the entries i of row s with first[s] <= i * page_size < end[s] let go of their pages
 * and become -1 (negative ones are passed over); a page without a holder goes back on the
 * stack.  Of the pages that go back, the one whose first entry comes first lies on top, so
 * that reserving the same entries again gives the same pages.  first = NULL: 0.
 *   - a sequence that ends: first NULL, end its length (or max_pages * page_size);
 *   - one that is cut back: first the new length, end the old one;
 *   - pages behind a window with first tokens that stay: first the sinks, end the window's first
 *     slot less page_size - 1.
 * An end above max_pages * page_size sets UP_DEVERR_BAD_KV_LENS and leaves the sequence out.  An
 * entry outside the pool (UP_DEVERR_BAD_PAGE), or of a page that nobody holds (any more:
 * UP_DEVERR_BAD_REFS), becomes -1 and nothing else happens to it.
 */
up_status up_release_pages(const up_page_pool *pool, int32_t *block_table, int num_seqs,
                           int max_pages, int page_size, const int32_t *first, const int32_t *end,
                           up_stream_t stream);

/*
 * Fork: child i (0 <= i < num_children) becomes a copy of sequence parents[i].  Its row of
 * table_out shares the parent's full pages (one holder more each); a partial last
 * page gets a free page of its own, whose rows up_copy_pages then copies in every layer's
 * cache.  Entries of the parent that are negative (released ones behind a window) stay -1, as
 * do those behind its kv_lens.
 *   table_out  int32 [num_children, max_pages].
 *   lens_out   int32 [num_children]: the parent's length.
 *   copies     int32 [3, num_children]: source page, new page, rows (-1, -1 where there is nothing
 *              to copy).
 * The three overlap neither one another nor block_table, kv_lens and parents (UP_ERR_INVALID_ARG).
 * A child whose parent is not in [0, num_seqs) (UP_DEVERR_BAD_TREE), has a length that cannot be
 * (UP_DEVERR_BAD_KV_LENS), or for which no free page is left (UP_DEVERR_NO_PAGES; earlier
 * children come first) is empty: length 0, no page.
 */
up_status up_fork_pages(const up_page_pool *pool, const int32_t *block_table,
                        const int32_t *kv_lens, int num_seqs, int max_pages, int page_size,
                        const int32_t *parents, int num_children, int32_t *table_out,
                        int32_t *lens_out, int32_t *copies, up_stream_t stream);

/*
 * Copies rows of pages, over all heads, in the keys, the values and (where the cache has them) the
 * positions: the first copies[2n + i] slots of page copies[i] to page copies[n + i].  A
 * negative page means nothing to copy.  No destination may be a source, or another copy's
 * destination.  A page outside the pool, or rows outside [0, page_size], set
 * UP_DEVERR_BAD_PAGE and copy nothing.  Of the cache the table and the lengths are not used.
 * Errors: UP_ERR_INVALID_ARG for a cache that the calls above do not take, or for more copies
 * than one launch has blocks (2 * Hk * ceil(page_size * d / 8192) * n below 2^31) or 32-bit
 * indexes reach (3 * n below 2^31).
 */
up_status up_copy_pages(const up_paged_kv *cache, const int32_t *copies, int num_copies,
                        up_stream_t stream);

/*
 * Instrumentation: when both events are non-NULL, every later scoring call
 * (up_score_blocks, up_score_blocks_shard, up_score_blocks_paged) made by this
 * host thread records `start_event` immediately before its
 * tensor-core scoring kernel and `stop_event` immediately after it, on the
 * call's stream, so the caller can time that kernel alone with
 * cudaEventElapsedTime.  Pass NULL, NULL to stop.  The events are cudaEvent_t
 * handles owned by the caller.  Not part of the method; no page counterpart.
 */
typedef struct CUevent_st *up_event_t;
up_status up_set_kernel_timing_events(up_event_t start_event, up_event_t stop_event);

/*
 * Instrumentation: measures this GPU's sustained MUFU ex2 rate (exponentials
 * per second over the whole device) with a short full-occupancy kernel on
 * `stream`, and writes it to *ex2_per_second.  Synchronises the stream (about
 * a millisecond).  This is the exponential roof of up_score_blocks, which
 * evaluates one ex2 per visible (query head, query, key) triple.  Not part of
 * the method; no page counterpart.
 */
up_status up_measure_ex2_rate(double *ex2_per_second, up_stream_t stream);

/*
 * Instrumentation for tests of the failure path: every spin-wait inside the
 * tensor-core scoring and attention kernels (a role waiting for shared-memory data,
 * a free TMEM buffer or another CTA's results) gives up after `cycles` SM clock
 * cycles; the kernel then stops every role of the CTA, lets its copies and
 * MMAs in flight complete, frees its tensor memory, returns and sets
 * UP_DEVERR_TIMEOUT (the call's outputs are then unspecified).  0 restores
 * the default bound (4e9 cycles, about two seconds); a bound above the
 * default returns UP_ERR_INVALID_ARG.  Process-wide; it applies to scoring
 * and attention calls issued after it.  Not part of the method; no page counterpart.
 */
up_status up_set_wait_limit(uint64_t cycles);

/*
 * Reads and clears the sticky device error word of the current device
 * (UP_DEVERR_* bits; 0 if none).  This call synchronises the device.
 * Returns UP_OK if no bit was set, UP_ERR_TIMEOUT if the timeout bit was set,
 * UP_ERR_DEVICE for any other bit, UP_ERR_CUDA if the copy itself failed.
 */
up_status up_get_device_error(uint32_t *bits);

#ifdef __cplusplus
}
#endif

#endif /* UP_H_ */
