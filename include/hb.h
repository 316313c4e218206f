/*
 * hb.h -- C ABI of the hybrid-batch paged-attention library (libhb.so).
 *
 * One call sequence runs one attention layer of a hybrid batch: many decode
 * rows (one new token each, over a long cached context) plus prefill chunks
 * (q_len > 1 new tokens that attend causally to themselves and re-read the
 * KV of the earlier chunks of their prompt), all over a paged KV cache.
 *
 *   hb_kv_append  scatter the batch's new K/V rows into their pages
 *   hb_plan       (host) split the batch into work items; upload the plan
 *   hb_attention  attention of every new token over its sequence's pages
 *
 * Around it, on the same batches: hb_linear (the block's projections), hb_norm,
 * hb_rope (in hb_kv_append's place for a model with rotary positions) and
 * hb_adapters; and, in their own sections, the 8-bit cache, pages on the GPU,
 * steps from host memory and the batch builder.
 *
 * The operation follows "Sarathi-Serve：以 chunked-prefills 与 stall-free batching
 * 驯服 LLM 推理的吞吐—延迟权衡", §GPU / 系统数据路径 ③ (a batch of decode tokens
 * plus prefill chunks within a token budget) and ⑤ (attention reads and
 * writes the KV cache through the page table; a chunk appends its KV, decodes
 * read all earlier KV, chunk i re-reads chunks 1..i-1), and "In-flight
 * Batching", §KV Cache 管理的协同优化 (16-token pages, a block table mapping
 * logical pages to non-contiguous physical ones) and §Batch 内的异构执行
 * (different lengths handled inside the kernel, no padding).
 *
 * Conventions shared by every call
 *  - Pointers are borrowed: the library allocates no device memory and keeps
 *    no pointer after the call returns (work already queued on `stream` uses
 *    them until it completes).  The caller owns all memory and streams.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default).
 *  - Argument errors are detected on the host and returned synchronously;
 *    nothing is launched then.  Device-side index errors (a block-table entry
 *    outside [0, num_pages)) set a device error word and skip the access;
 *    hb_check() turns it into HB_ERR_DEVICE_INDEX.  A device wait that runs
 *    out of time sets HB_ERR_TIMEOUT the same way.  No C++ exception crosses
 *    this boundary.  hb_last_error() gives a message for the last failure of
 *    the calling thread.
 *  - All calls are asynchronous on `stream` unless stated otherwise; append
 *    must be ordered before attention on the same stream.
 *  - The kernels are launched with programmatic stream serialization: a
 *    kernel of this library may start under the tail of the kernel before
 *    it and waits for that kernel before it depends on it.  When the
 *    library's previous launch on the stream is hb_kv_append of the same
 *    batch (same descriptors and pools), hb_attention waits for it only
 *    before reading the cache pages that hold the batch's new tokens and
 *    reads every other page at once; after anything else it waits first.
 *    Work of other libraries is complete before a kernel of this library
 *    starts (it does not release it early).
 *
 * Data layout (bf16 = IEEE bfloat16 stored as uint16)
 *  - q      [total_q, num_q_heads,  head_dim] bf16, rows in batch order
 *  - k_new  [total_q, num_kv_heads, head_dim] bf16 (same for v_new)
 *  - cache  [num_pages, page_size, num_kv_heads, head_dim] bf16, separate
 *           K and V pools ("NHD" pages)
 *  - out    [total_q, num_q_heads,  head_dim] bf16
 *  - Rows of sequence s are q rows cu_q_len[s] .. cu_q_len[s+1]-1.  Its new
 *    token j sits at logical position p = context_len[s] - q_len[s] + j in
 *    physical page block_table[s*max_pages_per_seq + p/page_size], slot
 *    p % page_size, and attends to logical keys 0..p (causal, aligned to the
 *    absolute position).  Query head h reads kv head h / (Hq/Hkv).
 *
 * Supported shapes: page_size 16, head_dim 64 or 128, Hq a multiple of Hkv
 * with group size Hq/Hkv <= 16, 1 <= q_len <= context_len per sequence (in the
 * 8-bit cache's calls and hb_pages_assign also q_len 0, a row that stands
 * still).
 */
#ifndef HB_H_
#define HB_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum hb_status {
  HB_OK = 0,
  HB_ERR_INVALID_ARG = 1,   /* null pointer, bad enum, misaligned pointer   */
  HB_ERR_SHAPE = 2,         /* inconsistent sizes or a row breaking          */
                            /* 1 <= q_len <= context_len                      */
  HB_ERR_UNSUPPORTED = 3,   /* valid but not built (page size, head_dim ...) */
  HB_ERR_WORKSPACE = 4,     /* plan or workspace buffer too small / stale    */
  HB_ERR_CUDA = 5,          /* a CUDA runtime/driver call failed             */
  HB_ERR_DEVICE_INDEX = 6,  /* a kernel met an out-of-range page index       */
  HB_ERR_TIMEOUT = 7,       /* a kernel wait gave up                         */
  HB_ERR_OUT_OF_PAGES = 8   /* batch builder: no free page for a decode;      */
                            /* hb_pages_assign: too few free pages            */
} hb_status;

/* Message for the last failed call on this thread ("" if none).  The string
 * is owned by the library and valid until the next call on this thread. */
const char* hb_last_error(void);

/* Name of a status code (static string). */
const char* hb_status_string(hb_status s);

/* Descriptor of one hybrid batch.  The three arrays are DEVICE pointers.
 *
 * sliding_window: 0 for full causal attention; W > 0 restricts the query at
 * absolute position p to the keys p-W+1 .. p (W keys, itself included).  The
 * pages name sliding-window model variants ("Sarathi-Serve: Chunked Prefills
 * for Stall-Free LLM Inference", §Results and evidence) without a size, so W
 * is a parameter.  With W > 0 the kernels never read the block-table entry
 * of a page that holds no key inside any of its row's windows (such entries
 * may be stale). */
typedef struct hb_batch {
  int32_t num_seqs;            /* sequences (rows of the batch), >= 0         */
  int32_t total_q;             /* sum of q_len = rows of q / k_new / out      */
  int32_t max_pages_per_seq;   /* row stride of block_table                   */
  int32_t num_pages;           /* physical pages in each cache pool           */
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t page_size;           /* tokens per page; must be 16                 */
  int32_t sliding_window;      /* 0: none; W > 0: keys p-W+1 .. p (above)     */
  int32_t reserved;            /* must be 0                                   */
  const int32_t* cu_q_len;     /* [num_seqs+1] prefix sums of q_len, [0] = 0  */
  const int32_t* context_len;  /* [num_seqs] tokens in cache AFTER append     */
  const int32_t* block_table;  /* [num_seqs * max_pages_per_seq] page ids     */
} hb_batch;

/*
 * KV append (scatter).  For every new token j of sequence s, copy row
 * cu_q_len[s]+j of k_new / v_new ([num_kv_heads*head_dim] contiguous bf16)
 * to its page slot in k_cache / v_cache (see the layout above).  The copy is
 * bit-exact; no other slot is written, and rows of k_new / v_new outside
 * every sequence's are written nowhere.  Cited passage: the first page,
 * §GPU / 系统数据路径 ⑤ ("a prefill chunk appends new KV").
 *   k_new, v_new     device, [total_q, Hkv, D] bf16, 16-byte aligned
 *   k_cache, v_cache device, [num_pages, 16, Hkv, D] bf16, 16-byte aligned
 * Errors: HB_ERR_INVALID_ARG / HB_ERR_SHAPE / HB_ERR_UNSUPPORTED on the host;
 * a page id outside [0, num_pages) is skipped and reported by hb_check().
 */
hb_status hb_kv_append(const hb_batch* batch, const void* k_new,
                       const void* v_new, void* k_cache, void* v_cache,
                       void* stream);

/*
 * Plan (host).  Cuts the batch into work items for hb_attention: decode rows
 * (q_len == 1) become split-KV items over page ranges, chunk rows (q_len > 1)
 * become (kv head, query tile) items; both lists are ordered longest first.
 * Needs HOST copies of q_len and context_len (the same values the device
 * arrays of `batch` hold) and the number of SMs of the device.
 *   h_q_len, h_context_len  host, [num_seqs] int32
 *   h_plan                  host buffer for the plan, or NULL
 *   plan_bytes              in: size of h_plan; out: bytes needed
 *   d_workspace             device buffer (256-byte aligned), or NULL
 *   workspace_bytes         in: size of d_workspace; out: bytes needed
 * The sizes are always reported.  With h_plan == NULL nothing else happens;
 * otherwise the plan is written into h_plan, and if d_workspace is not NULL
 * it is also copied into d_workspace and the workspace counters are cleared,
 * asynchronously on `stream` (only this step makes CUDA calls): h_plan must
 * stay unchanged until that copy has completed, and a workspace must not be
 * shared by attention calls in flight at once.  From pageable memory the
 * CUDA driver may wait for `stream` before it stages the copy: a caller
 * whose host should run ahead of the kernels passes a stream without the
 * previous step's kernels on it (for example its input-copy stream, ordered
 * before the kernels by an event).
 * The plan stays valid for any later hb_attention on a batch with the same
 * q_len / context_len / head geometry (block tables and tensors may change).
 * Errors: HB_ERR_SHAPE for rows outside 1 <= q_len <= context_len, or
 * context_len > max_pages_per_seq*page_size; HB_ERR_WORKSPACE if a buffer is
 * too small.
 */
hb_status hb_plan(const hb_batch* batch, const int32_t* h_q_len,
                  const int32_t* h_context_len, int32_t num_sms, void* h_plan,
                  size_t* plan_bytes, void* d_workspace,
                  size_t* workspace_bytes, void* stream);

/*
 * Attention.  out[row, h, :] = sum_t softmax_t(scale * <q[row,h], K[t]>) V[t]
 * over keys t = 0..p of the row's sequence (p its absolute position), K/V of
 * kv head h/(Hq/Hkv) read through the block table from the caches as they
 * stand after hb_kv_append.  fp32 accumulation, one bf16 rounding at the
 * store.  One kernel launch does all of it: decode rows are streamed as equal
 * page ranges per CTA (a row that straddles ranges leaves partial softmax
 * states, merged by the last piece to finish) and chunk rows are tiled for
 * the tensor cores, the two kinds of CTAs running side by side.
 * Cited passages: the first page, §GPU / 系统数据路径 ③-⑤, and §核心机制 3
 * (chunk i re-reads the KV of chunks 1..i-1; same computation as unchunked).
 *   h_plan      host plan written by hb_plan for this batch
 *   q, out      device, [total_q, Hq, D] bf16, 16-byte aligned
 *   k_cache, v_cache device pools as in hb_kv_append
 *   d_workspace the workspace hb_plan prepared
 * Errors: HB_ERR_WORKSPACE if h_plan does not match the batch; argument
 * errors as above; launch failures as HB_ERR_CUDA.
 */
hb_status hb_attention(const hb_batch* batch, const void* h_plan,
                       const void* q, const void* k_cache,
                       const void* v_cache, float softmax_scale, void* out,
                       void* d_workspace, void* stream);

/*
 * hb_attention, with the batch's new K/V rows also given as k_new / v_new
 * (the arrays passed to hb_kv_append for this batch, [total_q, Hkv, D] bf16,
 * 16-byte aligned).  The result is the same; the chunk rows read the pages
 * that hold only their sequence's new tokens from k_new / v_new instead of
 * from the caches, so they do not wait for the append kernel that writes
 * those pages (the one page holding a chunk's first token, when that token
 * does not start a page, and the decode rows' last pages are still read
 * from the caches after the append).  The caches must receive the new rows
 * by hb_kv_append as usual, queued before this call on the same stream.
 * Same passages as hb_attention.  Errors: as hb_attention;
 * HB_ERR_INVALID_ARG for a NULL or misaligned k_new / v_new.
 */
hb_status hb_attention_new_kv(const hb_batch* batch, const void* h_plan, const void* q,
                              const void* k_new, const void* v_new, const void* k_cache,
                              const void* v_cache, float softmax_scale, void* out,
                              void* d_workspace, void* stream);

/*
 * Decode attention without a workspace, for callers that cannot allocate
 * device memory.  (The pages have no counterpart of this call: it exists for
 * callers such as a serving engine that gives nearly all free HBM to its
 * KV-cache pool at start-up and allows no device allocation afterwards, or a
 * plugin that is handed raw tensor pointers but no allocator.)
 *
 * Same result as hb_plan + hb_attention on a batch whose rows are all decode
 * rows (q_len == 1), using the same split-KV kernel, but its scratch (work
 * items, counters, split partial states) is a fixed device array of
 * HB_NOALLOC_SCRATCH_BYTES inside the library, which every device that loads
 * the library holds until the process exits.  The call makes no cudaMalloc /
 * cudaFree and no other allocating call; its host-side plan also uses static
 * storage.  The caller still owns and passes q, the caches and out (layouts as
 * in hb_attention) plus host copies of q_len and context_len.
 *   - The first call on a device looks up that device's copy of the array
 *     (with the device current); make that first call before any stream
 *     capture.
 *   - All calls share the array and it keeps the last call's contents: each
 *     call clears the counters it needs; calls that overlap on the GPU (other
 *     streams or host threads) race and must be serialised by the caller.
 *     Host calls are serialised by a lock inside the library.
 *   - The plan's items are copied from pageable host memory, so the call
 *     returns after the copy is staged.  That storage is the library's own
 *     and the next call overwrites it, so a call on a stream that is being
 *     captured into a CUDA graph is refused with HB_ERR_UNSUPPORTED (a
 *     replayed copy would read a later call's items).
 *   - The work is spread over fewer CTAs when the partial states would not
 *     fit the array; a batch that needs more than 4096 work items (about
 *     num_seqs times ceil(Hkv / 8), plus one per SM) is rejected with
 *     HB_ERR_WORKSPACE.  Rows with q_len != 1 give HB_ERR_UNSUPPORTED.  Other
 *     errors as hb_attention.
 */
#define HB_NOALLOC_SCRATCH_BYTES (8u * 1024u * 1024u)

hb_status hb_decode_attention_noalloc(const hb_batch* batch,
                                      const int32_t* h_q_len,
                                      const int32_t* h_context_len,
                                      const void* q, const void* k_cache,
                                      const void* v_cache, float softmax_scale,
                                      void* out, void* stream);

/* ---------------------------------------------------------------------------
 * The 8-bit KV cache.  Half the bytes of the bf16 cache, for the same batch
 * descriptors, shapes (sliding windows included) and page layout:
 *   k_cache, v_cache device, [num_pages, 16, Hkv, D] e4m3 (the finite-only
 *                    8-bit float: 4 significant bits, +-448, NaN, no infinity),
 *                    16-byte aligned
 *   k_exp, v_exp     device, [num_pages, Hkv] int8: an element of page p and
 *                    kv head h stands for value * 2^exp[p, h]; exponents are
 *                    read as if held to [-64, 64]
 * Call order as with the bf16 cache: hb_kv8_append, then hb_kv8_attention
 * with a plan of hb_kv8_plan.  Cited passages as for hb_kv_append and
 * hb_attention (the pages do not speak of quantised caches).
 * ------------------------------------------------------------------------- */

/*
 * Quantising append.  For every page and kv head that receives new tokens,
 * with need = the smallest e in [-64, 64] such that the largest |x| of the
 * new finite elements is <= 448 * 2^e (-64 if they are all zero; 64 if none
 * reaches):
 *   - a page whose first slot is new gets exp = need; a page that holds older
 *     tokens of the sequence gets exp = max(its old exp, need), and if that
 *     grew, the older elements become round(value * 2^(old exp - exp));
 *   - a new element becomes round(x * 2^-exp), held to +-448; infinities and
 *     NaN become NaN and do not count towards need.
 * Rounding is to nearest even.  Other pages are not written; slots of a page
 * behind the sequence's last token keep their bytes.  A page must belong to
 * one sequence's new tokens only (a prefix may be shared between sequences
 * in whole pages that no batch row appends to).
 *   k_new, v_new     device, [total_q, Hkv, D] bf16, 16-byte aligned
 * Errors as hb_kv_append; HB_ERR_INVALID_ARG for NULL exponents,
 * HB_ERR_UNSUPPORTED for a batch of over 2^31 (page, head) pieces.
 */
hb_status hb_kv8_append(const hb_batch* batch, const void* k_new, const void* v_new,
                        void* k_cache, void* v_cache, int8_t* k_exp, int8_t* v_exp,
                        void* stream);

/* hb_plan for hb_kv8_attention (same arguments, rules and errors, but that a
 * row may also stand still: q_len 0 with any context_len, no row of q or out).
 * A plan serves one of the two: hb_attention refuses this one, hb_kv8_attention
 * refuses hb_plan's (HB_ERR_WORKSPACE).  The workspace also holds, if there is
 * a chunk row, the chunk rows' visible pages as bf16 (4 * Hkv * D bytes per
 * token, however few tokens the chunk has, and once for each row that shows a
 * shared page) and a block table of num_seqs * max_pages_per_seq entries: 32
 * rows of 16 tokens at a context of 8016 take 1 GB (8 heads of 128), twice
 * what their pages take in the cache.  A captured hb_kv8_attention reads the
 * plan in its workspace when it is replayed, so that workspace takes no other
 * plan meanwhile. */
hb_status hb_kv8_plan(const hb_batch* batch, const int32_t* h_q_len,
                      const int32_t* h_context_len, int32_t num_sms, void* h_plan,
                      size_t* plan_bytes, void* d_workspace, size_t* workspace_bytes,
                      void* stream);

/* hb_attention over the 8-bit cache: the same result, of the elements' values,
 * with the same masks and errors; HB_ERR_INVALID_ARG for a softmax_scale that
 * is not positive and finite.  Precision as hb_attention's, with two limits in
 * decode rows: a weight is rounded to 11 bits, but not finer than 2^-32 of the
 * row's largest weight, so a key below that counts with an error of up to that
 * part of its V; and of a row's pages (per kv head) those whose V scale is
 * over 2^64 below the largest may count as zeros.  What unwritten slots of a
 * page hold (NaN included) never shows, nor for a decode row what stands
 * below its window; a NaN stored as a value (V) of a chunk's own token may
 * reach the chunk's earlier rows too, as in hb_attention.  Work: decode rows
 * stream the 8-bit pages as they are; chunk rows' pages are spelt out as bf16
 * in the workspace by a launch before, and attended to as by hb_attention. */
hb_status hb_kv8_attention(const hb_batch* batch, const void* h_plan, const void* q,
                           const void* k_cache, const void* v_cache, const int8_t* k_exp,
                           const int8_t* v_exp, float softmax_scale, void* out,
                           void* d_workspace, void* stream);

/* ---------------------------------------------------------------------------
 * Page bookkeeping on the GPU: what hb_builder_* keeps on the host.  Tables,
 * prefix sums and free pages stay in device memory, where both appends (which
 * need nothing from the host) can follow in the same stream or graph; the
 * attention's plan still takes the lengths on the host.  slot_map is for a
 * caller's own scatter: the appends here go by block_table.  "In-flight
 * Batching", §KV Cache 管理的协同优化: fixed-size pages handed out as sequences
 * grow and freed when they finish.
 *
 * The free pages are a ring in device memory: free_pages [num_pages] int32
 * and a state of four int64: state[0] pages taken so far (head), state[1]
 * pages put in so far (tail), 0 <= head <= tail <= head + num_pages;
 * the free pages are free_pages[i % num_pages] for head <= i < tail, taken in
 * that order.  state[2] and state[3] are zero (a full pool starts as
 * free_pages = 0 .. num_pages-1, state = {0, num_pages, 0, 0}).  state_in is
 * read and state_out written (its four entries, whatever they held); both may
 * be the same array, and must not overlap otherwise (HB_ERR_INVALID_ARG).
 * Calls on one ring must be ordered.
 *
 * Lengths are read on the device, so mistakes in them are found there: the
 * call then takes and returns no page (state_out = state_in), and hb_check()
 * gives HB_ERR_SHAPE, or HB_ERR_OUT_OF_PAGES where only the free pages were
 * too few; what it leaves for the calls behind it, see below.  num_seqs is at
 * most 16384 (HB_ERR_UNSUPPORTED).
 * ------------------------------------------------------------------------- */

/*
 * For sequences with q_len[s] new tokens of context_len[s] after them (both
 * device int32, 0 <= q_len <= context_len <= max_pages_per_seq * 16; q_len 0:
 * a row that stands still):
 *   cu_q_len     [num_seqs+1] receives the prefix sums of q_len
 *   block_table  [num_seqs, max_pages_per_seq]: the entries of the logical
 *                pages that hold only new tokens, ceil((context_len - q_len)
 *                / 16) up to ceil(context_len / 16), receive pages from the
 *                ring, sequence by sequence in ascending order; the others
 *                stay as they are
 *   slot_map     [max_tokens] int64 or NULL: entry t receives page * 16 + slot
 *                of the t-th new token of the batch; entries behind the last
 *                token stay as they are
 * The sum of q_len must not exceed max_tokens.  A ring entry (or, for a token
 * on an older page, a table entry) outside [0, num_pages) becomes -1 and is
 * reported by hb_check() as HB_ERR_DEVICE_INDEX.
 * Behind a call that failed, calls already queued stay safe to run:
 *   - HB_ERR_SHAPE: no row has tokens by cu_q_len (all its entries equal the
 *     first, which stays) and no entry of slot_map is a slot (those >= 0 become
 *     -1), so an append writes nothing;
 *   - HB_ERR_OUT_OF_PAGES: cu_q_len is written, the tokens' slots are -1, and
 *     the table entries that were to receive pages name none (one in
 *     [0, num_pages) becomes -1, the others stay).  An append writes only to
 *     pages that the rows hold already, past their earlier tokens (there the
 *     8-bit scale may grow), and reports the others.  The same call again,
 *     with pages in the ring, fills the table as if it had been the first.
 */
hb_status hb_pages_assign(int32_t num_seqs, int32_t max_tokens, int32_t max_pages_per_seq,
                          int32_t num_pages, int32_t page_size, const int32_t* q_len,
                          const int32_t* context_len, const int32_t* free_pages,
                          const int64_t* state_in, int64_t* state_out, int32_t* block_table,
                          int32_t* cu_q_len, int64_t* slot_map, void* stream);

/*
 * The pages of finished sequences go back to the end of the ring: the first
 * ceil(lengths[s] / 16) entries of block_table row s, row by row in ascending
 * order (lengths: device int32, tokens in the cache, 0 for a row that keeps
 * its pages; the table is not changed).  Pages shared with a live sequence
 * must not be released.  HB_ERR_SHAPE by hb_check() if more come back than
 * were taken; a table entry outside [0, num_pages) is reported as
 * HB_ERR_DEVICE_INDEX and goes in as -1.
 */
hb_status hb_pages_release(int32_t num_seqs, int32_t max_pages_per_seq, int32_t num_pages,
                           int32_t page_size, const int32_t* lengths, const int32_t* block_table,
                           int32_t* free_pages, const int64_t* state_in, int64_t* state_out,
                           void* stream);

/* ---------------------------------------------------------------------------
 * One step from host memory.  For a serving loop that keeps a few steps in
 * flight: the step's inputs cross the host link as one packed block, the
 * plan goes up ahead of them on the input-copy stream, hb_kv_append and
 * hb_attention run on the compute stream, the output comes back on the
 * output-copy stream, and the step's slot (CUDA events and a device flag)
 * orders the three streams against the previous step that used the same
 * buffers.  The input copy is followed by a write of the step's sequence
 * number to the slot's flag, which the append kernel polls before it reads
 * its inputs (so the compute stream carries no wait between two steps and
 * each step's append launches under the previous attention's tail).  The
 * host does not wait, so one step's copies overlap the neighbouring steps'
 * kernels.  The operation is that of hb_kv_append then hb_attention (same
 * citations); only the copies and their ordering are added.
 *
 * Packed input block (host and device alike): q [total_q, Hq, D] bf16 |
 * k_new | v_new [total_q, Hkv, D] bf16 | cu_q_len [num_seqs+1] | context_len
 * [num_seqs] | block_table [num_seqs, max_pages_per_seq] int32, each section
 * starting on a 256-byte boundary.  hb_step_layout writes the six section
 * offsets and the block's size; it checks only the sizes it reads.
 * ------------------------------------------------------------------------- */
#define HB_STEP_SECTIONS 6

hb_status hb_step_layout(const hb_batch* shape, size_t offsets[HB_STEP_SECTIONS],
                         size_t* in_bytes);

/* Events and a 4-byte device flag of one set of staging buffers, on the
 * current device (creating a slot allocates the flag; destroying it frees
 * it, which synchronises the device). */
typedef struct hb_step_slot hb_step_slot;
hb_status hb_step_slot_create(hb_step_slot** out);
void hb_step_slot_destroy(hb_step_slot* slot);
/* Blocks until the slot's last step has completed (inputs consumed, output on
 * the host): call it before refilling the slot's host inputs or reading its
 * output. */
hb_status hb_step_slot_sync(hb_step_slot* slot);

typedef struct hb_step_buffers {
  const void* h_in;        /* host packed inputs (page-locked, for the copy to overlap) */
  void* d_in;              /* device packed inputs, 256-byte aligned                      */
  void* h_out;             /* host output [total_q, Hq, D] bf16                           */
  void* d_out;             /* device output, 16-byte aligned                              */
  void* h_plan;            /* host plan buffer (hb_plan's plan_bytes; page-locked makes   */
                           /* its upload asynchronous like the inputs')                    */
  size_t plan_bytes;
  void* d_workspace;       /* device workspace (hb_plan's workspace_bytes), 256-aligned   */
  size_t workspace_bytes;
} hb_step_buffers;

/*
 * The step.  `shape` gives the sizes (its three device pointers are ignored:
 * the descriptors are read from d_in); h_q_len / h_context_len are the host
 * copies hb_plan needs.  On copy_in_stream: wait for the slot's last kernels,
 * plan + upload (hb_plan), copy h_in -> d_in, raise the slot's flag.  On
 * stream: wait for the slot's last output copy if it is still pending when
 * the step is issued, hb_kv_append (which waits for the flag on the device,
 * bounded: a flag that does not come within about a second is reported as
 * HB_ERR_TIMEOUT by hb_check and the step's output is undefined),
 * hb_attention.  On copy_out_stream: wait for the kernels, copy d_out ->
 * h_out.  The buffers
 * belong to the slot until hb_step_slot_sync says its step is over; a slot's
 * buffers must not be shared with another slot.  The host blocks only if the
 * slot's previous input copy has not yet run (its plan buffer is rewritten
 * here).  Errors: as hb_plan, hb_kv_append and hb_attention;
 * HB_ERR_INVALID_ARG for NULL or misaligned buffers or a slot of another
 * device; HB_ERR_CUDA if an event or copy call fails.
 */
hb_status hb_step(const hb_batch* shape, const int32_t* h_q_len,
                  const int32_t* h_context_len, int32_t num_sms, hb_step_slot* slot,
                  const hb_step_buffers* buf, void* k_cache, void* v_cache,
                  float softmax_scale, void* copy_in_stream, void* stream,
                  void* copy_out_stream);

/*
 * Synchronise `stream`, then read and clear the device error word of the
 * current device: HB_OK, HB_ERR_DEVICE_INDEX or HB_ERR_TIMEOUT, after
 * hb_pages_* also HB_ERR_OUT_OF_PAGES or HB_ERR_SHAPE, which come before what
 * later calls reported because of them (or HB_ERR_CUDA if the stream itself
 * failed).  Blocking.
 */
hb_status hb_check(void* stream);

/*
 * Self-test of the failure path: launches one CTA that waits on a barrier
 * nothing arrives at, using the bounded wait every kernel of the library
 * uses.  After the wait's time limit (about one second) the kernel records a
 * timeout in the device error word and returns; hb_check() then gives
 * HB_ERR_TIMEOUT and the CUDA context stays usable.  No fault or hang.
 */
hb_status hb_selftest_wait_timeout(void* stream);

/*
 * The same for the flag wait of hb_step's append kernel (a device counter
 * that the input-copy stream raises): one CTA of two warps waits for a
 * device word that nothing raises; after the time limit each warp gives up,
 * the kernel records a timeout and returns, and hb_check() gives
 * HB_ERR_TIMEOUT.  No fault or hang.
 */
hb_status hb_selftest_flag_timeout(void* stream);

/* ---------------------------------------------------------------------------
 * Linear layer of a hybrid batch on the tensor cores: y = x W^T.  Cited
 * passage: the first page, §问题背景 (两阶段天然不对称) -- every token of the
 * batch also passes through the model's linear layers, which take most of
 * the iteration (compute-bound for prefill tokens, weight-read-bound for
 * decodes).  One persistent launch.
 *   x        device, [M, K] bf16 row-major (one row per token), 16-byte aligned
 *   w        device, [N, K] bf16 row-major (row n: weights of output n)
 *   M        rows (tokens), >= 0 (0: nothing to do)
 *   K        multiple of 64
 *   epilogue HB_LINEAR_STORE: y = x W^T, N a multiple of 256, its columns
 *              split over out->y[0..2] (out->cols[i] consecutive columns to
 *              y[i], each a multiple of 256 or 0, summing to N; y[i] is
 *              [M, cols[i]] row-major) -- e.g. q, k and v of a fused QKV
 *              projection;
 *            HB_LINEAR_GATED: w = [W_gate; W_up] with N = 2F rows (F a
 *              multiple of 128); y[0] [M, F] receives silu(x W_gate^T) *
 *              (x W_up^T), silu(g) = g / (1 + e^-g); cols[0] = F;
 *            HB_LINEAR_RESIDUAL: as STORE but y[i] += (its columns of)
 *              x W^T, in place (a residual connection).
 * Ownership: all pointers borrowed; nothing is allocated.  Errors:
 * HB_ERR_INVALID_ARG (NULL or misaligned pointer, unknown epilogue),
 * HB_ERR_SHAPE (sizes breaking the rules above); a wait that gives up is
 * reported by hb_check as HB_ERR_TIMEOUT.
 * ------------------------------------------------------------------------- */
typedef enum hb_linear_epilogue {
  HB_LINEAR_STORE = 0,
  HB_LINEAR_GATED = 1,
  HB_LINEAR_RESIDUAL = 2
} hb_linear_epilogue;

typedef struct hb_linear_out {
  void* y[3];          /* device, bf16; unused entries NULL                     */
  int32_t cols[3];     /* columns per destination (0 = unused)                 */
} hb_linear_out;

hb_status hb_linear(const void* x, const void* w, int32_t M, int32_t N, int32_t K,
                    int32_t epilogue, const hb_linear_out* out, void* workspace,
                    size_t workspace_bytes, void* stream);

/* Workspace that hb_linear can use for this problem on a device with num_sms
 * SMs (0: it needs none).  When the output tiles are too few to occupy the
 * SMs (few tokens), hb_linear splits each tile's K range over several CTAs;
 * the pieces meet in `workspace` (device, 256-byte aligned, ZERO-FILLED before
 * its first use; every call leaves it ready for the next, whatever its shape,
 * so one workspace of the largest size serves all problems).  With a NULL or
 * smaller workspace hb_linear runs unsplit.  Calls sharing a workspace must
 * not overlap on the GPU. */
size_t hb_linear_workspace_size(int32_t M, int32_t N, int32_t K, int32_t epilogue,
                                int32_t num_sms);

/* ---------------------------------------------------------------------------
 * Norms around the branches of a block.  (The pages name the block's linear
 * layers and its attention; its norms are what a model adds between them.)
 * For each of `rows` rows of `width` elements, with n(v, w) =
 * v * rsqrt(mean(v^2) + eps) * (weight_offset + w):
 *   u     = n(y, w_post), or y where w_post is NULL       the branch's output
 *   x_out = residual_scale * x + branch_scale * gate * u  the residual stream
 *   z     = n(x_out before its rounding, w_pre)           the next branch's input
 * Terms that are not given drop out: gate NULL counts as 1; without y the
 * stream is residual_scale * x (the first norm of a model), without x it is the
 * branch alone; w_pre NULL gives z without weights.  x or y, and x_out or z,
 * must be given; w_post and gate need y, w_pre needs z.
 *   y, gate, z       device, bf16
 *   w_post, w_pre    device, [width] bf16
 *   x, x_out         device, bf16 or fp32 (stream_type, both alike)
 *   *_stride         elements from row to row, 16 bytes a multiple;
 *                    gate_stride 0: one row of gates for all
 * width is a multiple of 8, at most 16384; pointers are 16-byte aligned.
 * x_out or z may be x, y or a gate per row, row for row and of the same
 * element size (in place), and overlap nothing otherwise
 * (HB_ERR_INVALID_ARG).  Sums and means are fp32 (64 bits where a row's
 * squares leave its range), one rounding per output; what stands between rows
 * is neither read nor written.  Many rows come by copies whose waits are
 * bounded; one that gives up is reported by hb_check as HB_ERR_TIMEOUT.
 * ------------------------------------------------------------------------- */
typedef enum hb_stream_type {
  HB_STREAM_BF16 = 0,
  HB_STREAM_FP32 = 1
} hb_stream_type;

typedef struct hb_norm_args {
  int32_t rows, width;
  int32_t stream_type;     /* hb_stream_type of x and x_out                  */
  int32_t reserved;        /* must be 0                                      */
  const void *x, *y, *gate, *w_post, *w_pre;
  void *x_out, *z;
  int64_t x_stride, y_stride, gate_stride, x_out_stride, z_stride;
  float eps;               /* >= 0                                           */
  float residual_scale, branch_scale, weight_offset;
} hb_norm_args;

hb_status hb_norm(const hb_norm_args* args, void* stream);

/* ---------------------------------------------------------------------------
 * Rotary positions.  (The pages leave a model's positions out; the attention
 * here takes q and k as they are, so this goes between the projection that
 * makes them and the append.)
 *
 * hb_rope_phases (host) writes the angle that pair i = 0 .. rotary_dim/2 - 1
 * of a head turns by from one position to the next, as a fraction of a turn in
 * 64-bit fixed point: phases[i] = f_i / (2 pi) * 2^64, with f_i = base^(-2 i /
 * rotary_dim) radians, scaled for contexts longer than the model was trained
 * on:
 *   HB_ROPE_PLAIN   f_i
 *   HB_ROPE_LINEAR  f_i / scale_by (positions interpolated)
 *   HB_ROPE_BASE    with base * scale_by^(rotary_dim / (rotary_dim - 2))
 *   HB_ROPE_PARTS   by frequency: a pair that makes t = original_context * f_i
 *                   / (2 pi) turns over the trained context keeps f_i from t =
 *                   high on, has f_i / scale_by up to t = low, and between
 *                   them f_i * (g + (1 - g) / scale_by), g = (t - low) / (high
 *                   - low): linear in t, not in the pair's index.  A model that
 *                   was trained with another ramp, or with a factor per pair,
 *                   needs phases of its own: hb_rope takes any
 * rotary_dim is a positive multiple of 16, base > 1, scale_by >= 1, 0 <= low <
 * high (what a kind does not use is not looked at).  64-bit arithmetic: a phase is
 * off by less than 2^-51 of a turn.
 * ------------------------------------------------------------------------- */
typedef enum hb_rope_scaling {
  HB_ROPE_PLAIN = 0,
  HB_ROPE_LINEAR = 1,
  HB_ROPE_BASE = 2,
  HB_ROPE_PARTS = 3
} hb_rope_scaling;

hb_status hb_rope_phases(int32_t rotary_dim, double base, int32_t scaling, double scale_by,
                         double original_context, double low, double high, uint64_t* phases);

typedef struct hb_rope_params {
  int32_t rotary_dim;      /* dims of a head that turn: a multiple of 16 in     */
                           /* [0, head_dim]; the others stay                    */
  int32_t interleaved;     /* 0: pair i is dims (i, i + rotary_dim/2); 1: (2i,  */
                           /* 2i+1)                                             */
  float factor;            /* multiplies what turns (an attention factor), or 1 */
  float eps;               /* of the head norms, >= 0                           */
  const uint64_t* phases;  /* device, [rotary_dim/2], 16-byte aligned           */
  const void* q_weight;    /* device, [head_dim] bf16: every q head is first    */
  const void* k_weight;    /* x * rsqrt(mean(x^2) + eps) * q_weight (k alike);  */
                           /* NULL: no such norm                                */
} hb_rope_params;

/*
 * For every new token of the batch, at its position p = context_len - q_len +
 * j: q and k heads normed (where weights are given) and turned by p, q into
 * q_out, k into k_out (unless NULL) and into its page slot of k_cache, v as it
 * is into its slot of v_cache (hb_kv_append's, which is then not needed).
 * Without caches (k_cache, v_cache and v all NULL) it only turns q and k, for
 * hb_kv8_append or an append elsewhere.  Tokens behind the last sequence are
 * left as they were; of the batch's descriptors, sliding_window plays no part.
 * fp32 arithmetic (a head whose squares leave its range is scaled for its
 * mean), one rounding.  An angle is position times phase modulo a turn, exact as
 * an integer at any position; it is off by 2^-26 of a turn at most where its
 * upper 32 bits become an fp32 number, and by the position times what the phase
 * itself is off (hb_rope_phases: less than 2^-51 of a turn).
 *   q, k, v          device, bf16: token rows of Hq * D and Hkv * D elements,
 *                    *_stride elements apart (a multiple of 8; larger than the
 *                    row where q, k and v are columns of one array)
 *   q_out, k_out     q and k themselves (in place, their strides), or [total_q,
 *                    heads, D] contiguous arrays that overlap no other operand
 *   k_cache, v_cache device pools as in hb_kv_append
 * Errors as hb_kv_append; HB_ERR_INVALID_ARG for operands that overlap.  A page
 * id outside [0, num_pages) is skipped (q_out and k_out are written) and
 * reported by hb_check().
 */
hb_status hb_rope(const hb_batch* batch, const hb_rope_params* rope, const void* q,
                  int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                  int64_t v_stride, void* q_out, void* k_out, void* k_cache, void* v_cache,
                  void* stream);

/* ---------------------------------------------------------------------------
 * Low-rank adapters of many requests beside a shared projection.  (The pages
 * serve one model to all requests; an adapter per request is what lets a
 * hybrid batch serve many models that share its weights.)  With adapter a of
 * the sequence that token t belongs to, for each destination i of hb_linear:
 *   out_i[t] = y_i[t] + scale[a] * (x[t] A_{a,i}^T) B_{a,i}^T
 * A pool holds the adapters of one projection:
 *   a      device, [num_adapters, slices, max_rank, K] bf16; slices = the
 *          projection's destinations (1 to 3), each with ranks of its own
 *   b      device, [num_adapters, N, max_rank] bf16, its rows as the
 *          projection's weight rows (destination by destination)
 *   rank   device, [num_adapters] int32: the ranks in use, read as if held to
 *          [0, max_rank]; what stands in a and b past them is not used
 *   scale  device, [num_adapters] fp32
 * max_rank is a multiple of 8, at most 128; K and each destination's columns are
 * multiples of 8.
 * ------------------------------------------------------------------------- */
typedef struct hb_adapter_pool {
  int32_t num_adapters, max_rank;
  int32_t K, N;            /* columns of x; columns of all destinations        */
  int32_t slices;          /* destinations                                     */
  const void *a, *b;       /* 16-byte aligned                                  */
  const int32_t* rank;
  const float* scale;
} hb_adapter_pool;

/*
 * Plan (host).  Sorts the batch's tokens by adapter: needs the host copies of
 * q_len (>= 0) and of each sequence's adapter (-1: none), and serves every pool
 * of num_adapters adapters with at most max_ranks = slices * max_rank ranks (all
 * projections of all layers of a step).  total_q: rows of x, y and out, at least
 * the sum of q_len; rows behind the last sequence are not written, and what a
 * tile's copies (whole boxes of 128 rows) read of them is not used.
 * Buffers, sizes and upload as with hb_plan (h_plan must stay unchanged until
 * its copy has completed; a workspace must not be shared by calls in flight at
 * once; a captured hb_adapters reads the plan in its workspace when it is
 * replayed, so that workspace takes no other plan meanwhile).  Runs of 128
 * neighbouring rows of an adapter or more (prompts) are cut into tiles of up to
 * 128 rows for the tensor cores, the other rows into segments of up to 16.  The
 * workspace also holds x A^T: for a tile's rows two bf16 terms (4 * (max_ranks +
 * 24) bytes each of 128 rows), for the others up to 16 parts in fp32 (4 *
 * max_ranks bytes per row and part; more parts where rows are few).
 * Errors: HB_ERR_SHAPE for lengths or adapters that break the rules,
 * HB_ERR_WORKSPACE if a buffer is too small.
 */
hb_status hb_adapters_plan(int32_t num_seqs, int32_t total_q, const int32_t* h_q_len,
                           const int32_t* h_adapter, int32_t num_adapters, int32_t max_ranks,
                           int32_t num_sms, void* h_plan, size_t* plan_bytes, void* d_workspace,
                           size_t* workspace_bytes, void* stream);

/*
 *   x        device, [total_q, K] bf16 (the projection's input), 16-byte aligned
 *   y, out   device, [total_q, cols[i]] bf16 each, columns alike; out may be y
 *            (in place, e.g. hb_linear's destinations), or arrays that overlap
 *            no other operand: rows whose sequence has no adapter are then
 *            copied.  out must not overlap x, nor the workspace any operand.
 * x A^T is summed in fp32 and enters the second product in two bf16 terms (16
 * bits); the sum with y is rounded once.  Two launches for the tiles and two for
 * the other rows, which run side by side.  A wait that gives up is reported by
 * hb_check as HB_ERR_TIMEOUT.  Errors:
 * HB_ERR_WORKSPACE if h_plan does not match the pool, HB_ERR_INVALID_ARG for
 * operands that overlap, others as hb_linear.
 */
hb_status hb_adapters(const hb_adapter_pool* pool, const void* h_plan, const void* x,
                      const hb_linear_out* y, const hb_linear_out* out, void* d_workspace,
                      void* stream);

/* ---------------------------------------------------------------------------
 * Instrumentation.  When enabled, every kernel launch of this library is
 * bracketed by CUDA events recorded on its launch stream.
 *   kernel ids: 0 = kv append (either cache), 1 = attention (decode and chunk
 *   work in one launch; over the 8-bit cache its widening launch is a record
 *   of its own), 2 = linear layer; the other calls are counted but not timed
 * ------------------------------------------------------------------------- */
#define HB_NUM_KERNEL_IDS 3

/* enable = 1: start recording, clearing earlier records; 2: resume
 * recording, keeping them (to time a sample of the launches); 0: stop (the
 * records stay readable).  Other values: HB_ERR_INVALID_ARG.  Not
 * thread-safe with concurrent launches from other threads. */
hb_status hb_timing_enable(int32_t enable);

/* Synchronise the recorded events and return, per kernel id, the summed
 * duration in milliseconds and the number of launches recorded.  Both arrays
 * have HB_NUM_KERNEL_IDS entries. */
hb_status hb_timing_read(double* total_ms, int32_t* launches);

/* Durations in milliseconds of the recorded launches of one kernel id, in
 * launch order: up to `max` of them go to ms[], *n receives how many were
 * recorded (which may exceed max).  Synchronises the events it reads. */
hb_status hb_timing_durations(int32_t kernel, float* ms, int32_t max, int32_t* n);

/* Number of kernels this library has launched in this process so far. */
int64_t hb_launch_count(void);

/* ---------------------------------------------------------------------------
 * Stall-free batch builder (host only, no CUDA).  Each step forms the next
 * hybrid batch: (1) one decode token of every request past its prefill,
 * (2) a chunk of every unfinished prefill, (3) first chunks of waiting
 * requests, first come first served, while the token budget lasts; then the
 * caller runs the batch and calls hb_builder_complete, which advances every
 * request and retires finished ones, returning their pages.  Cited passages:
 * the first page, §核心机制 2 (the four steps; decodes always in the batch,
 * at most B tokens per iteration); "In-flight Batching", §调度状态机 (waiting
 * -> prefill (chunked) -> decode -> completed).  Readings where the pages
 * are silent: chunk = min(prompt left, budget left); ongoing chunks shrink to
 * the pages available; admission stops at the first request whose first
 * chunk's pages cannot be allocated; pages come from the front of a FIFO free
 * list and return to its back; no preemption (a decode that finds no page
 * fails with HB_ERR_OUT_OF_PAGES); decodes that alone exceed the budget are
 * all kept and flagged over_budget.
 * ------------------------------------------------------------------------- */
typedef struct hb_builder hb_builder;

/* page_order: NULL for 0..num_pages-1, else a host permutation of it that
 * seeds the free list.  *out receives a new builder. */
hb_status hb_builder_create(int32_t budget, int32_t page_size,
                            int32_t num_pages, int32_t max_pages_per_seq,
                            const int32_t* page_order, hb_builder** out);
void hb_builder_destroy(hb_builder* b);

/* Queue a request (arrival order = call order).  HB_ERR_SHAPE if
 * prompt_len < 1, max_new < 1 or the request cannot fit max_pages_per_seq;
 * HB_ERR_INVALID_ARG for a duplicate id. */
hb_status hb_builder_add_request(hb_builder* b, int64_t id, int32_t prompt_len,
                                 int32_t max_new);

/* Form the next batch into caller-owned host arrays with room for max_rows
 * rows: q_len, context_len [max_rows], block_table [max_rows *
 * max_pages_per_seq] (unused entries -1), row_ids [max_rows], row_kind
 * [max_rows] (0 decode, 1 prefill).  *num_rows = 0 means nothing to run.
 * HB_ERR_WORKSPACE if max_rows is too small, HB_ERR_OUT_OF_PAGES if a
 * decode finds no free page; after any error the builder is unchanged.
 * A step costs what its rows and their pages cost, whatever the pool size.
 * Call hb_builder_complete before the next step. */
hb_status hb_builder_step(hb_builder* b, int32_t max_rows, int32_t* num_rows,
                          int32_t* q_len, int32_t* context_len,
                          int32_t* block_table, int64_t* row_ids,
                          int32_t* row_kind, int32_t* over_budget);

/* The batch of the last step ran.  Writes up to max_finished ids of the
 * requests that finished (in batch order) and their count. */
hb_status hb_builder_complete(hb_builder* b, int32_t max_finished,
                              int32_t* num_finished, int64_t* finished_ids);

/* Message for the last failed hb_builder_* call on this thread. */
const char* hb_builder_last_error(void);

/* Counts: waiting requests, running requests, free pages. */
hb_status hb_builder_counts(const hb_builder* b, int32_t* waiting,
                            int32_t* running, int32_t* free_pages);

/* The free list, front first (up to max entries; *n receives its length). */
hb_status hb_builder_free_list(const hb_builder* b, int32_t max, int32_t* n,
                               int32_t* pages);

#ifdef __cplusplus
}  /* extern "C" */
#endif

#endif  /* HB_H_ */
