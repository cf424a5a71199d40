/*
 * cpa.h -- C ABI of libcpa: one chunked-prefill attention step over a paged
 * KV cache, on one NVIDIA GB300 (sm_103a).
 *
 * The step ("vllm-learning-book 05. Chunked Prefill", sections 3 and 4):
 * a packed hybrid batch of S sequences whose scheduled tokens are concatenated
 * on one token axis with no padding.  Sequence s owns packed tokens
 * query_start_loc[s] .. query_start_loc[s+1]-1 (q_len of them) and holds
 * seq_lens[s] tokens in the cache once this step's K/V are appended.  A
 * prefill chunk has q_len > 1; a decode has q_len == 1.  Query row i of
 * sequence s attends to cache positions 0 .. seq_lens[s]-q_len+i: every
 * earlier chunk's K/V plus a causal mask inside the chunk (same page, Q&A of
 * section 8; "Chunked Prefill 技术深度解析", section 4.1).
 *
 * Conventions shared by every call
 *  - All pointers are device pointers unless a comment says otherwise.  The
 *    caller owns and allocates every buffer; the library never allocates
 *    device memory, never synchronises the stream, and keeps no state
 *    between calls besides the workspace the caller passes in.
 *  - Work is enqueued on `stream` (a cudaStream_t; NULL = legacy default
 *    stream) and runs asynchronously.
 *  - Arguments are validated on the host before anything is launched; an
 *    invalid argument returns a negative cpa_status and launches nothing.
 *  - Layouts (row-major, contiguous):
 *      q, out            [num_tokens][num_q_heads][head_dim]
 *      k, v (new tokens) [num_tokens][num_kv_heads][head_dim]
 *      k_cache, v_cache  [num_pages][num_kv_heads][page_size][head_dim]
 *      block_table       int32 [num_seqs][max_pages_per_seq]
 *      query_start_loc   int32 [num_seqs + 1], query_start_loc[0] == 0
 *      seq_lens          int32 [num_seqs]
 *      slot_mapping      int64 [num_tokens]
 *    Element type of q, k, v and out: `dtype` (fp32, bf16 or fp16).  The
 *    caches hold `dtype` too, or, with desc->kv_dtype = CPA_KV_E4M3 (16-bit
 *    dtypes only), one OCP FP8 E4M3 code per element (see cpa_kv_dtype).
 *  - GQA: query head h reads kv head h / (num_q_heads / num_kv_heads).
 *  - Supported: head_dim 64 or 128, page_size 16, num_q_heads a multiple of
 *    num_kv_heads with a group of 1, 2, 4 or 8 heads.
 */
#ifndef CPA_H
#define CPA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  CPA_OK = 0,
  CPA_ERR_ARG = -1,          /* malformed argument (null pointer, bad size)    */
  CPA_ERR_UNSUPPORTED = -2,  /* valid but not supported (e.g. head_dim 96)     */
  CPA_ERR_WORKSPACE = -3,    /* workspace missing, misaligned or too small     */
  CPA_ERR_CUDA = -4,         /* a CUDA runtime call or launch failed           */
  CPA_ERR_DEVICE = -5        /* a kernel found an out-of-range index or gave
                                up a bounded wait (status word, read back with
                                cpa_read_device_status)                       */
} cpa_status;

/* After CPA_ERR_DEVICE.  The word collects, since its last read, bit 1: a
 * block_table entry outside [0, num_pages) (that page was skipped), bit 2: a
 * slot_mapping entry past the cache (that row was not written), bit 4: a
 * bounded wait in the step kernel gave up (after 2^22 polls of its barrier,
 * on the order of a second; the CTA drained its copies and left, so some output rows of that call were
 * not written).  The output of every call since the last read is then
 * unreliable and must be recomputed; the cache rows the calls appended are
 * still valid unless bit 2 is set.  Nothing else needs resetting: the read
 * clears the word, and the next call rebuilds its work queue and zeroes its
 * counters itself.  Bits 1 and 2 mean the metadata is wrong; fix it before
 * re-running.  Bit 4 alone means the GPU did not run the kernel's CTAs to
 * completion in time (for instance a stream starved for longer than the wait
 * limit by other work); the same call can simply be issued again.
 * The page operators also raise bit 8: a row that could not be forked,
 * extended or released (left as it was), and bit 16: cpa_extend_sequences
 * found too few free pages (nothing was changed). */

typedef enum { CPA_F32 = 0, CPA_BF16 = 1, CPA_F16 = 2 } cpa_dtype;

/* Storage of the paged caches.
 *  CPA_KV_SAME  the caches hold `dtype` elements, bit for bit what was
 *               appended.
 *  CPA_KV_E4M3  the caches hold one byte per element: the OCP 8-bit floating
 *               point (OFP8) E4M3 code of the value divided by a per-tensor
 *               scale (desc->k_scale for K, desc->v_scale for V); the cached
 *               K is k_scale * E4M3 value, V likewise.  The append computes
 *               x / scale as one correctly rounded binary32 division, then
 *               rounds to the nearest E4M3 value (ties to even), saturating
 *               at +-448 (infinities included); NaN gives a NaN code.  The
 *               attention reads the codes exactly: the tensor cores multiply
 *               their exact binary16 values, q rounded to binary16 (exact for
 *               bf16 or fp16 inputs of magnitude 2^-17 .. 65504; larger
 *               magnitudes overflow), the softmax weights in binary16, with
 *               fp32 accumulation; k_scale is folded into the softmax scale
 *               and v_scale into the output.  Halves the cache bytes a step
 *               reads.  The pages do not cover an 8-bit cache: a library
 *               extension. */
typedef enum { CPA_KV_SAME = 0, CPA_KV_E4M3 = 1 } cpa_kv_dtype;

/* Problem description shared by the calls.  Sizes are host values. */
typedef struct cpa_desc {
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t page_size;
  int64_t num_pages;          /* pages in each of k_cache / v_cache           */
  int32_t max_pages_per_seq;  /* row stride of block_table; also bounds
                                 seq_lens[s] <= max_pages_per_seq * page_size */
  int32_t dtype;              /* cpa_dtype                                    */
  int64_t num_tokens;         /* packed tokens this step (query_start_loc[S]) */
  void *workspace;            /* device scratch, >= cpa_workspace_bytes(),
                                 256-byte aligned.  Only its first 4 bytes (the
                                 device status word) must be zero before the
                                 first call; every call resets the rest of the
                                 state it uses (work queue, merge counters),
                                 whatever an earlier call left there          */
  size_t workspace_bytes;
  int32_t kv_dtype;           /* cpa_kv_dtype; 0 = caches of `dtype`          */
  float k_scale, v_scale;     /* CPA_KV_E4M3: positive finite per-tensor
                                 scales; ignored otherwise                    */
} cpa_desc;

/* Human-readable name of a cpa_status value (static string, never NULL). */
const char *cpa_status_string(int status);

/* Bytes of workspace cpa_attention_forward needs for steps of at most
 * `num_seqs` sequences and desc->num_tokens packed tokens.  Pure host
 * arithmetic; returns 0 if the description is invalid.  The workspace holds
 * the step's work queue, the split-KV partial results (o, running max, running
 * sum) of decode segments and of chunk tiles split over several CTAs, their
 * arrival counters (zeroed by every call before use, never carried over from
 * an earlier call), and a device status
 * word.  It is sized for a GPU of up to 256 SMs. */
size_t cpa_workspace_bytes(const cpa_desc *desc, int32_t num_seqs);

/* KV append: for every packed token t with slot = slot_mapping[t] >= 0, copy
 * k[t][g][:] to k_cache[slot / page_size][g][slot % page_size][:] and likewise
 * v, for all kv heads g.  A negative slot skips the token.  The copy is
 * bit-exact (an E4M3 cache stores the codes of k / k_scale and v / v_scale,
 * see cpa_kv_dtype).  ("Chunked Prefill on an M5 Max", section "Wiring it into the
 * loop": a chunk extends the cache instead of rebuilding it; "Chunked Prefill
 * 技术深度解析", section 4.2: 16-token pages.)
 * Slots >= num_pages * page_size are skipped and raise the device status word
 * when a workspace is given in desc.  Tokens must map to distinct slots.
 * Only desc->num_kv_heads, head_dim, page_size, num_pages, dtype, num_tokens,
 * kv_dtype (with k_scale, v_scale) and (optionally) workspace are read. */
int cpa_kv_append(const void *k, const void *v, const int64_t *slot_mapping,
                  void *k_cache, void *v_cache, const cpa_desc *desc,
                  void *stream);

/* Attention forward of the whole hybrid batch in one call: out[t][h][:] =
 * softmax(scale * q[t][h] . K_j) . V_j over the visible cache positions j of
 * t's sequence (see the top of this file).  K/V are read through
 * block_table; the step's own new K/V must already be in the cache
 * (cpa_kv_append first).  Requires 1 <= q_len <= seq_lens[s] for every
 * sequence and seq_lens[s] <= max_pages_per_seq * page_size; entries of
 * block_table outside [0, num_pages) are not read and raise the device status
 * word.  Decodes with long contexts are split over the KV axis and merged in
 * the same launch with log-sum-exp weights ("Chunked Prefill 技术深度解析",
 * section 7.2: softmax normalised over the visible keys and combined
 * incrementally).  fp32 accumulation throughout; out has q's dtype.  With
 * fp32 activations the tensor cores round the chunk rows' MMA inputs to tf32
 * (10 mantissa bits); decode rows are computed in fp32 on CUDA cores. */
int cpa_attention_forward(const void *q, const void *k_cache, const void *v_cache,
                          const int32_t *block_table,
                          const int32_t *query_start_loc, const int32_t *seq_lens,
                          int32_t num_seqs, float scale, void *out, void *stream,
                          const cpa_desc *desc);

/* KV append and attention forward of one step in one call: the same results
 * as cpa_kv_append(k, v, slot_mapping, k_cache, v_cache, desc, stream)
 * followed by cpa_attention_forward(...) on the same stream -- the cache holds
 * the same bytes afterwards and out the same values -- without a separate
 * append launch ("Chunked Prefill on an M5 Max", section "Wiring it into the
 * loop": appending is part of each chunk's fixed cost).
 *  - Arguments: those of the two calls; k, v [num_tokens][Hkv][D] in the
 *    cache dtype and 16-byte aligned, slot_mapping int64 [num_tokens] and
 *    8-byte aligned.  slot_mapping[t] must be the cache slot of token t's
 *    position in its sequence (block_table[s][pos / 16] * 16 + pos % 16);
 *    tokens with a negative slot are not written, and no query may attend to
 *    them.
 *  - Where the step kernel takes the shape (bf16, head_dim 64 or 128, GQA
 *    group 1, 2, 4 or 8), the step's planning kernel copies the new rows into
 *    the cache while the attention kernel sets up, and the attention reads
 *    them from the cache once that copy is complete: a sequence may appear
 *    more than once in the batch (a chunk and a decode of the same sequence
 *    in one step).  Otherwise the call launches the append and then the
 *    attention on `stream`.
 *  - Errors: those of the two calls; slots >= num_pages * page_size raise the
 *    device status word and are not written. */
int cpa_append_attention_forward(const void *q, const void *k, const void *v,
                                 const int64_t *slot_mapping, void *k_cache, void *v_cache,
                                 const int32_t *block_table, const int32_t *query_start_loc,
                                 const int32_t *seq_lens, int32_t num_seqs, float scale,
                                 void *out, void *stream, const cpa_desc *desc);

/* ---- Attention with a sliding window and sinks ------------------------------
 * The pages have no counterpart to these calls, nor to the page operators
 * below: library extensions for serving with a bounded cache.
 *
 * The query row at position x of its sequence (x = seq_lens[s] - q_len + i for
 * row i) sees cache position j when j <= x and (j < sinks or j > x - window):
 * the last `window` positions, its own among them, and the first `sinks`
 * positions, which stay visible for good.  Everything else is as in
 * cpa_attention_forward: the whole packed batch of chunks and decodes, every
 * dtype and cache storage, the workspace (cpa_workspace_bytes), the arguments'
 * checks, and the status word.
 *  - window >= 1 (so no row is without a visible key), sinks >= 0; CPA_ERR_ARG
 *    otherwise.  A window of at least the context is plain causal attention.
 *    max_pages_per_seq * page_size is at most 2^30 (CPA_ERR_UNSUPPORTED).
 *  - The cost is that of the visible keys, whatever the length of the sequence.
 *    Only pages that hold a position some row of the sequence sees are looked
 *    up and read: block_table entries of the others may be anything (pages
 *    given back with cpa_release_pages have -1 there).
 *  - Keys and values no row of a 256-row group (256 / G consecutive tokens of a
 *    chunk; a decode on its own) sees may hold anything, NaN included.  Inside
 *    a chunk a non-finite V that one row of the group sees can make the outputs
 *    of the group's other rows non-finite, as in cpa_attention_forward.
 *  - fp32 activations keep fp32's precision: the tensor cores multiply each
 *    operand as the sum of two tf32 values, the products' error is below
 *    2^-21 (cpa_attention_forward rounds a chunk's operands to tf32).  There a
 *    non-finite q, K or V that a row sees gives non-finite outputs: NaN
 *    where the formula's value is infinite, and where it is finite because the
 *    key's score is -infinity.  A magnitude of (2 - 2^-11) 2^127 and more, which is
 *    infinite in tf32, counts as not finite. */
int cpa_window_attention_forward(const void *q, const void *k_cache, const void *v_cache,
                                 const int32_t *block_table, const int32_t *query_start_loc,
                                 const int32_t *seq_lens, int32_t num_seqs, float scale,
                                 int32_t window, int32_t sinks, void *out, void *stream,
                                 const cpa_desc *desc);

/* cpa_kv_append and cpa_window_attention_forward of one step in one call, as
 * cpa_append_attention_forward is of cpa_attention_forward: the same results
 * as the two calls, fused where the step kernel takes the shape. */
int cpa_append_window_attention_forward(const void *q, const void *k, const void *v,
                                        const int64_t *slot_mapping, void *k_cache, void *v_cache,
                                        const int32_t *block_table,
                                        const int32_t *query_start_loc, const int32_t *seq_lens,
                                        int32_t num_seqs, float scale, int32_t window,
                                        int32_t sinks, void *out, void *stream,
                                        const cpa_desc *desc);

/* ---- Page operators --------------------------------------------------------
 * Sequences that share pages, and a pool whose pages are given back, on the
 * device: no call waits for the host, and all can be captured into a graph.
 *
 * State (device memory, the caller's):
 *   block_table  int32 [num_rows][max_pages_per_seq]; entry c of a row holds
 *                positions 16 c .. 16 c + 15, -1 (any negative value) where
 *                the row holds no page
 *   seq_lens     int32 [num_rows]
 *   page_refs    int32 [num_pages], 16-byte aligned: how many block_table
 *                entries hold the page; 0 = free
 * block_table and seq_lens are those of the attention calls.  The results
 * depend on the state alone: where pages are chosen, the lowest are taken, and
 * rows count in their order.  One table and one page_refs may serve the caches
 * of many layers: the table operators move no K or V, they list the copies to
 * make, and cpa_copy_pages makes them, once per layer.
 * The table operators read desc->num_pages, page_size (16), max_pages_per_seq
 * (at most 2^26) and workspace: at least cpa_pages_workspace_bytes, 256-byte
 * aligned, its first four bytes (the status word, cpa_read_device_status) zero
 * before the first use.  Calls that may overlap on the GPU need workspaces of
 * their own.  num_pages is below 2^27. */

/* Workspace of the table operators for a pool of num_pages; 0 if out of range. */
size_t cpa_pages_workspace_bytes(int64_t num_pages);

/* For every pair i < n: page src[i] of k_cache and of v_cache is copied, bit
 * for bit, to page dst[i].  n is max_pairs, or, with num_pairs not NULL, the
 * device value *num_pairs (at most max_pairs count).  The pages in dst are
 * distinct, and none of them is in src (the lists of cpa_extend_sequences and
 * cpa_compact_pages are so); where they are not, those pages' contents are
 * unspecified.  A pair that names a page outside [0, num_pages) is skipped and
 * raises the status word when a workspace is given in desc.  Reads the cache's
 * shape and type from desc, as cpa_kv_append does; max_pairs may be 0. */
int cpa_copy_pages(const int32_t *src, const int32_t *dst, const int32_t *num_pairs,
                   int32_t max_pairs, void *k_cache, void *v_cache, const cpa_desc *desc,
                   void *stream);

/* For every fork i: row children[i] becomes a copy of row parents[i], the
 * length with it, and every page it holds gains a reference.  No page is
 * copied, the partly filled last one neither: cpa_extend_sequences does that
 * when one of its holders writes to it.  A parent may be forked many times.
 * A child's row holds no page before the call, is no other child of the call
 * and no parent in it; a fork whose child is not so, or with a row outside
 * [0, num_rows), is left out whole and raises the status word.  At most 4096
 * forks per call (CPA_ERR_UNSUPPORTED), and no more than num_rows. */
int cpa_fork_sequences(const int32_t *parents, const int32_t *children, int32_t num_forks,
                       int32_t *block_table, int32_t *seq_lens, int32_t num_rows,
                       int32_t *page_refs, const cpa_desc *desc, void *stream);

/* Makes room for a step's new tokens, which are described as for the attention
 * calls: row s takes q_len = query_start_loc[s + 1] - query_start_loc[s] tokens
 * (0: none), and seq_lens[s] counts them already.  In the order of the rows,
 * and of the pages in each:
 *  - where the new tokens have no page, the row takes the lowest page that was
 *    free before the call;
 *  - where the first of them goes to a page that holds earlier tokens and other
 *    references, the row gives its reference up, takes the lowest free page
 *    instead, and the pair (old, new) is listed in copy_src, copy_dst.  If all
 *    of a page's references are rows that write to it so, the last of them
 *    keeps it;
 *  - where a page for new tokens alone (the row was set back to a shorter
 *    length, say) has other references, the row gives its reference up and takes
 *    the lowest free page; there is nothing to copy;
 *  - slot_mapping[t] is the slot of every new token t, as cpa_kv_append and
 *    the fused attention calls take it.
 * counts (int32 [2], device): the number of pairs listed, and of pages taken.
 * The pairs have to be copied (cpa_copy_pages with num_pairs = counts, in every
 * layer's cache) before the step's rows are appended.
 * If fewer pages are free than the step needs, nothing is changed: every
 * slot_mapping entry is -1, counts = {0, -needed} (at least -2^31 + 1), and the
 * status word is raised.  (The attention calls take rows with tokens only: a caller whose rows
 * sit steps out gathers the others' block_table, query_start_loc and seq_lens.)
 * A row with q_len < 0, seq_lens[s] < q_len, more tokens than its
 * block_table row or than desc->num_tokens can hold takes nothing, its tokens'
 * slots are -1, and the status word is raised; so is it by an entry past the
 * pool.  Tokens past the last row's have slot -1.
 * num_seqs rows of block_table, at most 4096 (CPA_ERR_UNSUPPORTED);
 * slot_mapping int64 [desc->num_tokens]; copy_src, copy_dst int32 [num_seqs],
 * written up to the count. */
int cpa_extend_sequences(const int32_t *query_start_loc, const int32_t *seq_lens,
                         int32_t num_seqs, int32_t *block_table, int32_t *page_refs,
                         int64_t *slot_mapping, int32_t *copy_src, int32_t *copy_dst,
                         int32_t *counts, const cpa_desc *desc, void *stream);

/* Gives pages of num_released rows back (rows: their numbers; NULL: rows 0 ..
 * num_released - 1): the entries become -1 and their pages lose a reference.
 *  - window >= 1: the pages that no query from position seq_lens[row] on sees
 *    with this window and sinks (see cpa_window_attention_forward): those
 *    wholly at or behind `sinks` and wholly before seq_lens[row] - window + 1.
 *  - window = 0 (sinks = 0): every page; seq_lens[row] becomes 0.
 * A row may be named twice.  A row outside [0, num_rows) is left out and
 * raises the status word, as does an entry whose page is past the pool or
 * counts as free. */
int cpa_release_pages(const int32_t *rows, int32_t num_released, int32_t *block_table,
                      int32_t *seq_lens, int32_t num_rows, int32_t window, int32_t sinks,
                      int32_t *page_refs, const cpa_desc *desc, void *stream);

/* Packs the pool: afterwards its m live pages are pages 0 .. m - 1.  The j-th
 * free page below m takes the place of the j-th live page from m on; page_refs
 * and every entry of block_table (all rows that hold pages of the pool) follow,
 * and the pairs (old, new) are listed in
 * copy_src, copy_dst (int32 [num_pages / 2] each, written up to the count), to
 * be copied in every layer's cache before anything reads or writes it.
 * counts (int32 [2], device): the number of pairs, and m.  An entry whose page
 * counts as free or is past the pool stays as it is and raises the status
 * word.  Any number of rows. */
int cpa_compact_pages(int32_t *block_table, int32_t num_rows, int32_t *page_refs,
                      int32_t *copy_src, int32_t *copy_dst, int32_t *counts,
                      const cpa_desc *desc, void *stream);

/* Size of the scratch array built into the library for
 * cpa_attention_forward_noalloc: 64 MiB of device memory on every GPU that
 * loads the library, held until the process exits. */
#define CPA_NOALLOC_SCRATCH_BYTES (64u << 20)

/* CPA_NOALLOC_SCRATCH_BYTES as the library was built with it (for bindings
 * that cannot read the macro). */
size_t cpa_noalloc_scratch_bytes(void);

/* Attention forward for callers that may not allocate device memory.  The
 * pages have no counterpart to this call: it is a library convenience.
 * Callers in this position include plugins inside a host runtime that owns
 * all device memory and passes in only inputs and outputs, and serving loops
 * that forbid cudaMalloc/cudaFree after start-up because those calls can
 * synchronise the device and can fail under memory pressure mid-step.
 *
 * Same computation, arguments and layouts as cpa_attention_forward, except
 * that desc->workspace and desc->workspace_bytes are ignored: the scratch
 * lives in a fixed array compiled into the library.  The call allocates
 * nothing (no cudaMalloc, no cudaFree, no allocating library routine).
 *  - Limit: the workspace this step would need, cpa_workspace_bytes(desc,
 *    num_seqs), must not exceed CPA_NOALLOC_SCRATCH_BYTES; larger steps are
 *    rejected with CPA_ERR_WORKSPACE before anything is launched.
 *  - Set-up: every call looks up the array's device address in the current
 *    context with cudaGetSymbolAddress (host-side; nothing is allocated).
 *    The first call in a context may load the library's device code, so make
 *    it before any stream capture.  CPA_ERR_CUDA if the lookup fails.
 *  - Sharing: every call on a device uses the same array, which keeps what the
 *    last call left in it.  Once a call has passed its argument checks it
 *    clears the array's status word on `stream`, right before its first
 *    launch (the call resets its work queue and merge counters itself); a
 *    rejected or empty call touches nothing.
 *    Calls whose work overlaps on the GPU (different streams, or different
 *    host threads) race on the array: serialise them.
 *  - Errors: those of cpa_attention_forward; out-of-range indices met by the
 *    kernels are reported by cpa_noalloc_read_device_status. */
int cpa_attention_forward_noalloc(const void *q, const void *k_cache, const void *v_cache,
                                  const int32_t *block_table,
                                  const int32_t *query_start_loc, const int32_t *seq_lens,
                                  int32_t num_seqs, float scale, void *out, void *stream,
                                  const cpa_desc *desc);

/* Synchronously read (and clear) the device status word of the no-alloc
 * scratch array on the current device: CPA_OK, or CPA_ERR_DEVICE if the last
 * cpa_attention_forward_noalloc call on this device met an out-of-range page
 * index or gave up a bounded wait (its output is then incomplete).  Waits for
 * `stream`; allocates nothing.  Test/debug helper, not meant for the hot
 * path.  Returns CPA_ERR_ARG for a null status_out, CPA_ERR_CUDA if a CUDA
 * call fails. */
int cpa_noalloc_read_device_status(void *stream, int32_t *status_out);

/* Synchronously read (and clear) the device status word held in the
 * workspace: CPA_OK, or CPA_ERR_DEVICE if a kernel since the last read met an
 * out-of-range page or slot index.  Waits for `stream`.  Test/debug helper,
 * not meant for the hot path. */
int cpa_read_device_status(const cpa_desc *desc, void *stream, int32_t *status_out);

#ifdef __cplusplus
}
#endif

#endif /* CPA_H */
