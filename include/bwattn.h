/*
 * libbwattn: exact scaled-dot-product attention on one GB300 (sm_103a).
 *
 *   O = softmax(Q K^T * scale) V,  scale normally 1/sqrt(d)
 *
 * computed with the online-softmax recurrence (a running max m, running sum l and an
 * unnormalised output o, rescaled by exp(m - m_new) tile by tile), so that the score matrix
 * never reaches device memory. Sources, by page title and section:
 *   - "Attention from the kernel's side: FlashAttention, online softmax and fused dequant":
 *     "The online softmax" (the recurrence), "FlashAttention: what never touches memory"
 *     (Q tile resident, K/V tiles streamed, O written once), "Prefill and decode are
 *     different problems" (GQA reuse, flash-decoding split over the KV axis).
 *   - "Attention kernels" (llm-inference-explained): "Maths" (the recurrence and the merge
 *     rule for two partial states (m, l, o)), "Concept" (split-K decode).
 *   - "Attention Computation in Practice": section 5, "The four attention kernels you
 *     actually use" (prefill, decode, append/mixed with cu_seqlens, cross attention),
 *     "GQA in the kernel" (query head h reads KV head h / (Hq / Hkv)), "Masking variants"
 *     (causal j <= i and the skip / full / diagonal rule per block pair).
 *
 * Conventions shared by every call:
 *   - Every tensor pointer is a DEVICE pointer owned by the caller, contiguous in the layout
 *     given (calls with stride arguments: in those strides), 16-byte aligned (int32 arrays and lse:
 *     their own size; attn_fwd_host alone takes host pointers). The library never
 *     allocates or frees memory and never synchronises the host.
 *   - Every call is asynchronous on `stream` (a cudaStream_t passed as void*; NULL = the
 *     legacy default stream) and returns a status code. Argument checks happen on the host
 *     before any CUDA call, so a rejected call has no side effect.
 *   - Causal masking with Nq != Nk is aligned to the end: query i sees key j iff
 *     j <= i + (Nk - Nq). A query that sees no key gets O = 0 and LSE = -inf.
 *   - LSE (log-sum-exp) is the natural log of sum_j exp(scale * q.k_j) over the visible keys,
 *     written as fp32. Passing lse = NULL skips it.
 *   - Inputs are bf16 (IEEE bfloat16) unless a dtype argument says otherwise; arithmetic is
 *     fp32 (tensor cores with fp32 accumulation for bf16 inputs, fp32 FMA for fp32 inputs).
 *   - State kept across calls: a device status word that records a timed-out internal wait
 *     (see bwattn_get_status); rings of per-launch device counters (the prefill's item
 *     counters, the decode's merge tickets), each launch taking its share when it is enqueued
 *     and leaving it reset; the static scratch of attn_decode_static; the streams and events
 *     of attn_fwd_host. Calls are thread-safe and may be captured into CUDA graphs (except
 *     attn_fwd_host).
 *   - Limit of those rings, per device: a share is handed out again after 4096 further
 *     prefill launches (item counters) or 65,536 further merge tickets (a fused-merge decode
 *     takes one ticket per (sequence, KV head, row group)). Calls still running when their
 *     share comes round again would share it and corrupt each other's scheduling or merge:
 *     keep fewer launches than that in flight on one device at a time, counting every replay
 *     of a captured graph that runs concurrently with other calls.
 */
#ifndef BWATTN_H
#define BWATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ---- */
#define BWATTN_OK 0
#define BWATTN_ERR_INVALID_ARG 1 /* null pointer, size out of range, Hq % Hkv != 0, misaligned pointer, workspace too small */
#define BWATTN_ERR_UNSUPPORTED 2 /* valid arguments outside what the kernels implement (dtype / head dim / group size) */
#define BWATTN_ERR_CUDA 3        /* a CUDA runtime call or kernel launch failed; see bwattn_last_cuda_error() */
#define BWATTN_ERR_TIMEOUT 4     /* a kernel gave up an internal wait; reported by bwattn_get_status() */

/* ---- dtypes ---- */
#define BWATTN_DTYPE_FP32 0
#define BWATTN_DTYPE_BF16 1

/*
 * attn_fwd: prefill / cross attention over dense batches.
 * ("Attention Computation in Practice", section 5, kernel classes 1 and 4;
 *  "Attention from the kernel's side", "FlashAttention: what never touches memory".)
 *
 *   q, o : [B, Hq, Nq, d]        (dtype; o has the same dtype as q)
 *   k, v : [B, Hkv, Nk, d]       (dtype)
 *   lse  : [B, Hq, Nq] fp32, may be NULL
 *   causal: 0 = no mask (cross attention), 1 = causal aligned to the end
 *   scale: multiplies q.k before the softmax; must be finite and > 0
 *   dtype: BWATTN_DTYPE_BF16 (tcgen05 tensor-core kernel, d in {64, 128, 256}: the fast
 *          kernels' head dims, "Production implications"; d = 256 keeps one query tile per
 *          CTA because its fp32 O tile fills half of tensor memory) or
 *          BWATTN_DTYPE_FP32 (fp32 FMA kernel, d in {64, 128})
 * Query head h reads KV head h / (Hq / Hkv). Nq = 0 or B = 0 is a valid no-op; Nk = 0 gives
 * O = 0 and LSE = -inf. Errors: INVALID_ARG for null / misaligned pointers, negative sizes,
 * Hq % Hkv != 0, bad scale; UNSUPPORTED for other d or dtype.
 */
int attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv, int Nq,
             int Nk, int d, int causal, float scale, int dtype, void* stream);

/*
 * attn_fwd_host: attn_fwd on HOST-resident tensors (same shapes, layouts, dtypes and errors),
 * copies included. The (sequence, KV head) units are cut into up to 8 chunks; each chunk's
 * copies in, kernel and copies out run on library-owned streams so that transfers overlap
 * kernels (no counterpart on the pages; it is the host-memory end of the same computation).
 *
 *   q, k, v, o, lse : HOST pointers in the attn_fwd layouts; page-locked memory is needed for
 *                     the copies to overlap (pageable memory works, serialised); lse may be NULL
 *   workspace       : DEVICE buffer, 256-byte aligned, of at least
 *                     attn_fwd_host_workspace_size(B, Hq, Hkv, Nq, Nk, d, dtype) bytes (two
 *                     chunks of staging); contents undefined on exit
 *   stream          : the work starts after everything already queued on it, and work queued on
 *                     it afterwards starts after the last copy out; the host buffers must stay
 *                     valid until then
 * Calls from several host threads are serialised while they enqueue (the streams are shared).
 * On an error return after copies were queued (a CUDA error part way through), the call first
 * waits on the host for its own streams, so no copy from or to the host buffers is still
 * running when it returns; the outputs are then undefined.
 */
int attn_fwd_host(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv, int Nq,
                  int Nk, int d, int causal, float scale, int dtype, void* workspace, size_t workspace_bytes,
                  void* stream);
size_t attn_fwd_host_workspace_size(int B, int Hq, int Hkv, int Nq, int Nk, int d, int dtype);

/*
 * attn_fwd_window: causal prefill with a sliding window ("Attention Computation in Practice",
 * "Masking variants": sliding window i - W < j <= i). Same layouts, dtypes and errors as
 * attn_fwd with causal = 1; query i sees keys j with i' - window < j <= i', i' = i + (Nk - Nq).
 * K/V tiles entirely outside every row's window are not read. window >= 1, else INVALID_ARG;
 * window >= Nk gives the plain causal result.
 */
int attn_fwd_window(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv, int Nq,
                    int Nk, int d, int window, float scale, int dtype, void* stream);

/*
 * attn_decode_workspace_size: bytes of caller-provided workspace attn_decode needs for the
 * per-split partial states (m, l, o[d]) in fp32.
 */
size_t attn_decode_workspace_size(int B, int Hq, int d, int num_splits);

/*
 * attn_decode: single-query decode against a contiguous KV cache, split over the KV axis
 * (flash-decoding), partial states merged with the two-state merge rule.
 * ("Attention from the kernel's side", "Prefill and decode are different problems";
 *  "Attention kernels", "Maths", second display; "Attention Computation in Practice",
 *  section 5, kernel class 2 and "PagedAttention's kernel difference", contiguous form.)
 *
 *   q, o     : [B, Hq, d] bf16 (the one new query of each sequence)
 *   kcache,
 *   vcache   : [B, Hkv, nk_cap, d] bf16
 *   nk       : [B] int32 DEVICE array, valid keys per sequence, 0 <= nk[b] <= nk_cap;
 *              every valid key is visible (the new token's K/V are already in the cache)
 *   num_splits: KV slices per (sequence, KV head), 1..1024; slices past nk[b] are empty
 *   scale    : finite, > 0
 *   lse      : [B, Hq] fp32, may be NULL
 *   workspace: device buffer of at least attn_decode_workspace_size(B, Hq, d, num_splits)
 *              bytes; contents on entry are ignored, on exit undefined. Must not be shared
 *              by calls that may overlap on the GPU.
 * The g = Hq / Hkv query heads of a group are packed against each K/V tile, so every cache
 * byte is read once. Supported: d in {64, 128, 256} ("Production implications": the fast
 * kernels' head dims), 1 <= g <= 32. Errors as for attn_fwd, plus INVALID_ARG when the
 * workspace is NULL or too small.
 */
int attn_decode(const void* q, const void* kcache, const void* vcache, void* o, const int32_t* nk, int B, int Hq,
                int Hkv, int nk_cap, int d, int num_splits, float scale, float* lse, void* workspace,
                size_t workspace_bytes, void* stream);

/*
 * attn_decode_paged: single-query decode against a paged KV cache: the cache is a pool of
 * fixed-size pages and a per-sequence block table lists which page holds each run of
 * page_size consecutive keys. ("Attention Computation in Practice", "PagedAttention's kernel
 * difference": block_table[b] = [17, 3, 92, ...], read block 17, then 3, ...; the kernel takes
 * the table as an argument and gathers.) Same split-K pass and merge as attn_decode.
 *
 *   q, o        : [B, Hq, d] bf16
 *   k_pages,
 *   v_pages     : [num_pages, page_size, Hkv, d] bf16 (a page holds page_size consecutive keys
 *                 of every KV head)
 *   block_table : [B, max_pages_per_seq] int32 DEVICE array; key j of sequence b is row
 *                 j % page_size of page block_table[b][j / page_size]. Entries outside
 *                 [0, num_pages) are clamped into the pool (wrong data, never an out-of-bounds read)
 *   nk          : [B] int32 DEVICE array, 0 <= nk[b] <= max_pages_per_seq * page_size
 *   page_size   : a multiple of 16, 16..1024
 *   workspace   : at least attn_decode_workspace_size(B, Hq, d, num_splits) bytes
 * Supported: d in {64, 128, 256}, 1 <= g <= 32. Errors as for attn_decode.
 */
int attn_decode_paged(const void* q, const void* k_pages, const void* v_pages, void* o, const int32_t* block_table,
                      const int32_t* nk, int B, int Hq, int Hkv, int page_size, int num_pages, int max_pages_per_seq,
                      int d, int num_splits, float scale, float* lse, void* workspace, size_t workspace_bytes,
                      void* stream);

/*
 * attn_decode_fp8 / attn_decode_paged_fp8: attn_decode / attn_decode_paged against an FP8 KV
 * cache, each code turned into its value inside the kernel as it is loaded ("Attention from the
 * kernel's side", "Why a quantised cache needs a fused kernel": a separate dequantise pass would
 * move more bytes than the 16-bit cache it replaces; rule 3 of "Rules I use"). The pages' own
 * format (TBQ4) belongs to another project; this is the generic FP8 form:
 *
 *   kcache, vcache /
 *   k_pages, v_pages : the layouts of attn_decode / attn_decode_paged with one byte per element,
 *                      an OCP FP8 E4M3 code (bias 7, no infinities, S.1111.111 = NaN, max 448)
 *   k_scale, v_scale : [Hkv, d] fp32 DEVICE arrays, 16-byte aligned; the cached value of channel
 *                      c of KV head h is e4m3(code) * k_scale[h * d + c] (v_scale for V)
 *   q, o, lse, nk, block_table, page_size, num_splits, scale, workspace: as for attn_decode /
 *                      attn_decode_paged (same workspace size)
 * The cache is read exactly once; arithmetic is f16 x f16 products of the codes against
 * q * k_scale (rescaled per query row by a power of two) with fp32 accumulation. Supported:
 * d = 128, 1 <= g <= 32. Errors as for attn_decode, plus INVALID_ARG for NULL or unaligned
 * scales.
 */
int attn_decode_fp8(const void* q, const void* kcache, const void* vcache, const float* k_scale,
                    const float* v_scale, void* o, const int32_t* nk, int B, int Hq, int Hkv, int nk_cap, int d,
                    int num_splits, float scale, float* lse, void* workspace, size_t workspace_bytes, void* stream);

int attn_decode_paged_fp8(const void* q, const void* k_pages, const void* v_pages, const float* k_scale,
                          const float* v_scale, void* o, const int32_t* block_table, const int32_t* nk, int B, int Hq,
                          int Hkv, int page_size, int num_pages, int max_pages_per_seq, int d, int num_splits,
                          float scale, float* lse, void* workspace, size_t workspace_bytes, void* stream);

/*
 * attn_decode_static: the same single-query split-K decode as attn_decode, for callers that
 * cannot allocate device memory. The pages have no counterpart to this entry point; it exists
 * for deployment. Some callers cannot call cudaMalloc or hand the library a workspace: a
 * plugin or inference-engine host that gives a kernel only its input and output buffers, code
 * whose device memory is entirely owned by another allocator, or a latency-critical loop that
 * cannot afford cudaMalloc's implicit device-wide synchronisation. This call takes the same
 * arguments as attn_decode minus the workspace, and keeps its per-split partial states in a
 * fixed array of BWATTN_DECODE_STATIC_SCRATCH_BYTES inside the library, which every GPU that
 * loads the library holds until the process exits. It allocates nothing.
 *   - Limit: the partials must fit the array, i.e.
 *     attn_decode_workspace_size(B, Hq, d, num_splits) <= BWATTN_DECODE_STATIC_SCRATCH_BYTES
 *     (about B * Hq * num_splits <= 16,000 at d = 128); larger calls return
 *     BWATTN_ERR_UNSUPPORTED without launching anything.
 *   - The first call on each device looks up the array's device address (once per device,
 *     with that device current); make that first call before any stream capture.
 *   - Every call on a device shares the one array, and the array keeps the last call's
 *     contents. Nothing in it needs to start at zero (each call writes every partial it later
 *     reads), but calls that overlap on the GPU (other streams, other host threads) race on it:
 *     order them, e.g. on one stream.
 * Errors otherwise as for attn_decode.
 */
#define BWATTN_DECODE_STATIC_SCRATCH_BYTES (8u * 1024u * 1024u)
int attn_decode_static(const void* q, const void* kcache, const void* vcache, void* o, const int32_t* nk, int B,
                       int Hq, int Hkv, int nk_cap, int d, int num_splits, float scale, float* lse, void* stream);

/*
 * attn_varlen_workspace_size: bytes of workspace attn_varlen needs, from the host-side
 * bounds it is given.
 */
size_t attn_varlen_workspace_size(int num_seqs, int max_seqlen_k, int Hq, int Hkv, int d);

/*
 * attn_varlen: packed batches of sequences with different lengths (append / mixed:
 * speculative verify, chunked prefill), described by prefix sums of the lengths.
 * ("Attention Computation in Practice", section 5, kernel class 3, "varlen kernels with
 *  cu_seqlens".)
 *
 *   q, o         : [total_q, Hq, d] bf16, sequence s owns rows cu_seqlens_q[s] .. cu_seqlens_q[s+1]-1
 *   k, v         : [total_k, Hkv, d] bf16, sequence s owns rows cu_seqlens_k[s] .. cu_seqlens_k[s+1]-1
 *   total_q,
 *   total_k      : host-side row counts of the packed tensors (= cu_seqlens_*[num_seqs]); they
 *                  bound every tensor-core load, so no copy ever reads past the buffers
 *   lse          : [total_q, Hq] fp32, may be NULL
 *   cu_seqlens_q,
 *   cu_seqlens_k : [num_seqs + 1] int32 DEVICE arrays, non-decreasing, [0] = 0
 *   max_seqlen_q,
 *   max_seqlen_k : host-side upper bounds of the per-sequence lengths (grid sizing); a
 *                  sequence longer than its bound is not processed correctly
 *   causal       : 1 = causal aligned to each sequence's end, 0 = none
 *   workspace    : device buffer of at least attn_varlen_workspace_size(...) bytes
 * Sequences whose n_q * (Hq / Hkv) <= 32 run on the split-K decode kernel (all query heads
 * of a KV group packed in one tile); the others run on the tcgen05 prefill kernel. When both
 * run, the split-K pass is a programmatic dependent launch that starts on the SMs the prefill
 * leaves; it still completes after the prefill, so work queued on `stream` after the call sees
 * the whole output.
 * Supported: d in {64, 128, 256}, 1 <= g <= 32. Errors as for attn_decode.
 */
int attn_varlen(const void* q, const void* k, const void* v, void* o, float* lse, const int32_t* cu_seqlens_q,
                const int32_t* cu_seqlens_k, int num_seqs, int total_q, int total_k, int max_seqlen_q,
                int max_seqlen_k, int Hq, int Hkv, int d, int causal, float scale, void* workspace,
                size_t workspace_bytes, void* stream);

/*
 * attn_varlen_window: attn_varlen with causal = 1 and a sliding window of `window` keys ending
 * at each query's causal limit (aligned to each sequence's end). window >= 1, else INVALID_ARG.
 */
int attn_varlen_window(const void* q, const void* k, const void* v, void* o, float* lse, const int32_t* cu_seqlens_q,
                       const int32_t* cu_seqlens_k, int num_seqs, int total_q, int total_k, int max_seqlen_q,
                       int max_seqlen_k, int Hq, int Hkv, int d, int window, float scale, void* workspace,
                       size_t workspace_bytes, void* stream);

/* ---- speculative decoding over a cache: drafted token trees, paged plans and appends ---- */

/*
 * attn_tree_workspace_size: bytes of workspace attn_tree / attn_tree_paged need, from the
 * host-side bounds they are given (0 for sizes they refuse).
 */
size_t attn_tree_workspace_size(int num_seqs, int max_nodes, int Hq, int Hkv, int d);

/*
 * attn_tree / attn_tree_paged: verification of drafted token trees. The queries of a sequence are
 * the nodes of its tree; each sees every context key of the sequence's cache and those drafted
 * tokens of its own sequence that its mask names (its ancestors and itself, for a tree), whose
 * keys and values are read from the packed k_new, v_new and need not be in the cache. (The pages'
 * append class, "Attention Computation in Practice", section 5, kernel class 3, covers drafts that
 * form one line; the mask takes the place of its causal rule.)
 *
 *   q, o         : [total_q, Hq, d] bf16, sequence s owns nodes cu_seqlens_q[s] .. cu_seqlens_q[s+1]-1;
 *                  consecutive nodes of q lie q_stride elements apart (heads d apart; o is contiguous)
 *   k_new, v_new : [total_q, Hkv, d] bf16, the nodes' own keys and values, consecutive nodes
 *                  k_new_stride / v_new_stride elements apart (slices of a fused projection's rows)
 *   kcache, vcache / k_pages, v_pages, block_table : the cache in the layouts of attn_decode /
 *                  attn_decode_paged (kcache, vcache may be NULL when nk_cap is 0)
 *   nk           : [num_seqs] int32 DEVICE array, context keys per sequence, 0 <= nk[s] <= nk_cap (or
 *                  max_pages_per_seq * page_size); all of them are visible to every node
 *   cu_seqlens_q : [num_seqs + 1] int32 DEVICE array, non-decreasing, [0] = 0; rows of q behind
 *                  cu_seqlens_q[num_seqs] belong to no sequence, their o and lse are left as they were
 *   mask         : [total_q, ceil(max_nodes / 64)] uint64 DEVICE array: bit j % 64 of word j / 64 of a
 *                  node's row is set iff the node sees draft j of its sequence; bits at or past the
 *                  sequence's node count are ignored. A node that sees no key gets O = 0, LSE = -inf
 *   total_q      : host-side row count of the packed tensors
 *   max_nodes    : host-side upper bound of the nodes of a sequence, at most 1024; a longer
 *                  sequence's further nodes are neither read nor written
 *   lse          : [total_q, Hq] fp32, may be NULL
 *   workspace    : at least attn_tree_workspace_size(...) bytes; contents undefined on exit. Must not
 *                  be shared by calls that may overlap on the GPU
 * Keys and values that a node does not see (context rows at or past nk, drafts its mask leaves out)
 * have no effect on its outputs, whatever they hold (infinities and NaN included). Scores, the sum of the
 * weights and O are held in fp32; each weight is rounded to bf16 (by at most 2^-8 of itself) for the product
 * with V, as attn_fwd's are. Supported: d in
 * {64, 128, 256}, Hq / Hkv <= 128, max_nodes <= 1024. Strides are multiples of 8 and at least
 * Hq * d (q) or Hkv * d (k_new, v_new), else INVALID_ARG; other errors as for attn_decode.
 */
int attn_tree(const void* q, const void* kcache, const void* vcache, const void* k_new, const void* v_new, void* o,
              float* lse, const int32_t* nk, const int32_t* cu_seqlens_q, const uint64_t* mask, int num_seqs,
              int total_q, int max_nodes, int nk_cap, int Hq, int Hkv, int d, int64_t q_stride, int64_t k_new_stride,
              int64_t v_new_stride, float scale, void* workspace, size_t workspace_bytes, void* stream);

int attn_tree_paged(const void* q, const void* k_pages, const void* v_pages, const int32_t* block_table,
                    const void* k_new, const void* v_new, void* o, float* lse, const int32_t* nk,
                    const int32_t* cu_seqlens_q, const uint64_t* mask, int num_seqs, int total_q, int max_nodes,
                    int page_size, int num_pages, int max_pages_per_seq, int Hq, int Hkv, int d, int64_t q_stride,
                    int64_t k_new_stride, int64_t v_new_stride, float scale, void* workspace, size_t workspace_bytes,
                    void* stream);

/*
 * attn_tree_mask: the masks and positions of drafted trees from their parent links.
 *
 *   parents      : [total_q] int32, the parent of node i of a sequence as an index within the sequence;
 *                  parents come before their children: a value outside [0, i) makes node i a root
 *   cu_seqlens_q : as for attn_tree
 *   nk           : [num_seqs] int32 context keys, or NULL (0 for every sequence)
 *   mask         : [total_q, ceil(max_nodes / 64)] uint64, written: bit j of node i's row is set iff j
 *                  is i or an ancestor of i
 *   positions    : [total_q] int32, written unless NULL: nk[s] + depth of the node (0 for a root)
 * Rows that belong to no sequence, and nodes past a sequence's first max_nodes, are left as they were.
 */
int attn_tree_mask(const int32_t* parents, const int32_t* cu_seqlens_q, const int32_t* nk, uint64_t* mask,
                   int32_t* positions, int num_seqs, int total_q, int max_nodes, void* stream);

/*
 * kv_plan_paged: room in a paged cache for n_new[b] further tokens of each request b: pages from a
 * stack of free ones, the block table extended by them, and the slot of every new token. ("Attention
 * Computation in Practice", "PagedAttention's kernel difference": the block table that the paged
 * kernels read.) All arrays are int32 DEVICE arrays.
 *
 *   nk, n_new   : [B] keys that request b has in the cache, and tokens to make room for (negative: 0)
 *   held        : [B] pages that request b holds: block_table[b][0 .. held[b]-1]. It may hold more
 *                 than its keys fill (room left by drafts that were not accepted)
 *   free_pages,
 *   free_count  : [free_capacity], [1]: a stack of free pages; the last of the first *free_count is taken first
 *   block_table : [B, max_pages_per_seq], extended in place: with need_b = max(0, min(ceil((nk + n_new) /
 *                 page_size), max_pages_per_seq) - held), request b's entries held .. held + need_b - 1
 *                 become the next need_b pages of the stack, request after request. Other entries stay
 *   nk_out, held_out : [B] nk + n_new; held + need_b
 *   cu_seqlens  : [B + 1] exclusive prefix sums of n_new (the total last)
 *   slots       : [num_tokens] slot of the j-th new token of request b at cu_seqlens[b] + j: page *
 *                 page_size + row of position nk[b] + j. -1 behind the last token and where there is no
 *                 page: the stack ran out, or the position is past max_pages_per_seq pages
 *   free_count_out : [1] *free_count less the pages taken; negative by how many the stack was short,
 *                 whose table entries are -1: nothing of the plan may then be used, release pages and
 *                 plan again
 * The outputs must not overlap the inputs (equal pointers: INVALID_ARG). page_size is a multiple of 16,
 * 16..1024, B * max_pages_per_seq below 2^31. The call may be repeated on the same inputs with the same
 * results.
 */
int kv_plan_paged(const int32_t* nk, const int32_t* n_new, int32_t* block_table, const int32_t* held,
                  const int32_t* free_pages, const int32_t* free_count, int32_t* nk_out, int32_t* held_out,
                  int32_t* cu_seqlens, int32_t* slots, int32_t* free_count_out, int B, int page_size,
                  int max_pages_per_seq, int free_capacity, int num_tokens, void* stream);

/*
 * kv_append_paged / kv_append_paged_fp8: new K and V rows written into the pages at given slots.
 *
 *   k_new, v_new : [num_rows, Hkv, d] bf16, consecutive rows k_new_stride / v_new_stride elements apart
 *   slots        : [num_slots] int32 DEVICE array, the pool row (page * page_size + row of the page)
 *                  that slot i writes; values outside [0, num_pages * page_size) are skipped
 *   rows         : [num_slots] int32 DEVICE array, the row of k_new and v_new that slot i takes (the
 *                  accepted nodes of a verified tree); values outside [0, num_rows) are skipped. NULL:
 *                  slot i takes row i (num_slots <= num_rows)
 *   k_pages,
 *   v_pages      : [num_pages, page_size, Hkv, d]: bf16 for kv_append_paged; one E4M3 code per
 *                  element for kv_append_paged_fp8, the layout of attn_decode_paged_fp8
 *   k_scale,
 *   v_scale      : [Hkv, d] fp32 DEVICE arrays, 16-byte aligned, positive and normal: the code of a value x is the
 *                  E4M3 code nearest to x / scale (ties to the even code; magnitudes past 448, infinities
 *                  among them, become +-448; NaN stays NaN)
 * Slots must differ from one another: of two slots with one value, which row stays is not defined (and
 * may differ within the row). k_new and v_new may be rows of the pools themselves if no row that is read
 * is also written. Supported: d in {64, 128, 256}. num_slots = 0 or num_rows = 0 is a no-op.
 */
int kv_append_paged(const void* k_new, const void* v_new, const int32_t* slots, const int32_t* rows, void* k_pages,
                    void* v_pages, int num_slots, int num_rows, int page_size, int num_pages, int Hkv, int d,
                    int64_t k_new_stride, int64_t v_new_stride, void* stream);

int kv_append_paged_fp8(const void* k_new, const void* v_new, const int32_t* slots, const int32_t* rows,
                        void* k_pages, void* v_pages, const float* k_scale, const float* v_scale, int num_slots,
                        int num_rows, int page_size, int num_pages, int Hkv, int d, int64_t k_new_stride,
                        int64_t v_new_stride, void* stream);

/* ---- status and diagnostics ---- */

/* The cudaError_t of the last failing CUDA call made by this thread inside the library (0 if none). */
int bwattn_last_cuda_error(void);

/* Short text for a status code (static storage). */
const char* bwattn_status_string(int status);

/*
 * bwattn_get_status: synchronises `stream`, then returns BWATTN_ERR_TIMEOUT if any kernel of
 * this library on the current device gave up an internal wait since the last
 * bwattn_clear_status(), else BWATTN_OK (or BWATTN_ERR_CUDA if the synchronisation failed).
 * A kernel that gives up a wait writes no further output and leaves the context usable.
 */
int bwattn_get_status(void* stream);

/* bwattn_clear_status: resets the device status word (ordered on `stream`). */
int bwattn_clear_status(void* stream);

/*
 * bwattn_set_wait_timeout_ns: the bound on any single internal wait of a kernel (default
 * 2e9 ns); applies to launches made after the call, from any thread.
 */
void bwattn_set_wait_timeout_ns(uint64_t ns);

/*
 * bwattn_test_wait_timeout: launches a one-CTA kernel that waits on a barrier nothing ever
 * arrives at, bounded by the current wait timeout, so a test can check that a timed-out wait
 * returns BWATTN_ERR_TIMEOUT through bwattn_get_status() with the context still usable.
 */
int bwattn_test_wait_timeout(void* stream);

/* Number of kernels this library has launched successfully in this process (all threads). */
uint64_t bwattn_launch_count(void);

/* Library version, major * 10000 + minor * 100 + patch. */
int bwattn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* BWATTN_H */
