// Internal launch interface between the C-ABI layer (api.cu) and the kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace bw {

constexpr float kLog2e = 1.4426950408889634f;
// Bit of the device status word (owned by the C-ABI layer, passed to kernels as a pointer)
// that records a wait some kernel gave up.
constexpr unsigned int kStatusTimeoutBit = 1u;
constexpr float kLn2 = 0.6931471805599453f;

// ---- fp32 FMA prefill (any B, heads, lengths; d in {64, 128}) ----
struct Fp32FwdArgs {
  const float* q;
  const float* k;
  const float* v;
  float* o;
  float* lse;
  int B, Hq, Hkv, Nq, Nk, d, causal;
  float scale_log2;  // scale * log2(e)
  int window;        // > 0: sliding window of that many keys ending at the causal limit
};
cudaError_t launch_prefill_fp32(const Fp32FwdArgs& a, cudaStream_t stream);

// ---- split-K pass over the KV axis (decode and small-n_q varlen sequences) ----
// A "unit" is (sequence, KV head, row group); its rows are the (query, head) pairs
// r = i * g + hh of that sequence's queries and the group's query heads, group_rows (8 or 16)
// per row group.
struct SplitKArgs {
  const uint16_t* q;  // bf16 bits; token-major [tokens, Hq, D]
  const uint16_t* k;  // bf16 bits
  const uint16_t* v;
  float* ws;          // partials: (m, l) then o, see splitk_ws_layout()
  const int32_t* nk;  // dense decode: [B] valid keys per sequence (device)
  const int32_t* cu_q;  // varlen: [num_seqs + 1] (device), else null
  const int32_t* cu_k;
  int num_seqs, Hq, Hkv, g;
  int d;              // head dim D: 64 or 128 (128 with an FP8 cache)
  int64_t kv_seq_stride;  // dense: elements between sequences' caches (Hkv * cap * D)
  int64_t kv_head_stride;  // elements between KV heads at the same key (dense: cap * D, varlen: D)
  int64_t kv_key_stride;   // elements between consecutive keys (dense: D, varlen: Hkv * D)
  int kv_cap;         // dense: cache capacity (nk[b] is clamped to it)
  int total_q, total_k;  // varlen: rows of the packed tensors (cu_seqlens are clamped to them)
  int num_splits;
  int rows_max;       // workspace rows per (sequence, KV head)
  int group_rows;     // rows per row group: 8 (transposed 8-row MMA form) or 16 (16-row form)
  int row_groups;     // ceil(rows_max / group_rows)
  int causal;         // varlen: causal aligned to each sequence's end
  int window;         // varlen: > 0 adds a sliding window of that many keys
  int small_rows_limit;  // varlen: a sequence takes this path iff n_q * g <= this
  int min_chunk;         // varlen: a split takes at least this many keys (a multiple of 16; 0: none)
  size_t ws_o_offset;    // splitk_o_offset(num_seqs * Hkv, num_splits, rows_max)
  float scale_log2;
  // paged KV cache (decode only) when block_table is non-null: k, v are [num_pages, page_size,
  // Hkv, D]; key j of sequence b lives in page block_table[b * max_pages + j / page_size],
  // row j % page_size (page_size a multiple of 16, so a 16-key step never crosses a page)
  const int32_t* block_table;
  int page_size, max_pages, num_pages;
  // FP8 KV cache when k8 is non-null (k, v unused): E4M3 codes laid out like k, v; the value of
  // element (head h, channel c) is e4m3(code) * k_scale[h * D + c] (v_scale for V). tm_k8 and
  // tm_v8 are 3-D uint8 maps with a 128-byte swizzle whose box is one 16-key step of one KV
  // head: contiguous {128, cap, B * Hkv}, box {128, 16, 1}; paged {128, Hkv, pages * page_size},
  // box {128, 1, 16}
  CUtensorMap tm_k8, tm_v8;
  // bf16 16-row form at d = 128 (contiguous or packed cache, no window) when tma16 is non-zero:
  // K and V rows arrive by TMA through tm_k16 / tm_v16, 3-D bf16 maps with a 128-byte swizzle
  // whose box is 16 keys x 64 channels of one KV head: contiguous {128, cap, B * Hkv}, box
  // {64, 16, 1}; packed {128, Hkv, total_k}, box {64, 1, 16}
  CUtensorMap tm_k16, tm_v16;
  int tma16;
  const uint8_t* k8;
  const uint8_t* v8;
  const float* k_scale;
  const float* v_scale;
  // fused merge when tickets is non-null: units * row_groups zeroed counters owned by this
  // launch (left zeroed again); the last CTA of each (unit, row group) writes o and lse
  unsigned int* tickets;
  uint16_t* o;
  float* lse;
  // the FP8 instances' copies are waited for with a bounded wait (timeout_ns); one that gives up
  // sets kStatusTimeoutBit in *status (the device status word)
  unsigned int* status;
  uint64_t timeout_ns;
  // varlen: non-zero when the call's prefill kernel was launched just before on the same stream.
  // The pass reads nothing that kernel writes, so it is then a programmatic dependent launch whose
  // CTAs take the SMs the prefill's persistent CTAs leave; its last CTA waits for the prefill grid
  // to complete, so that this grid (and the work queued after it) completes after the prefill
  int after_prefill;
};
cudaError_t launch_splitk(const SplitKArgs& a, cudaStream_t stream);

struct MergeArgs {
  const float* ws;
  uint16_t* o;  // bf16 bits, token-major [tokens, Hq, D]
  float* lse;   // [tokens, Hq] or null
  const int32_t* cu_q;  // varlen or null (dense: one token per sequence)
  const int32_t* cu_k;
  const int32_t* nk;
  int num_seqs, Hq, Hkv, g, num_splits, rows_max, small_rows_limit;
  int d;  // head dim: 64 or 128
  int total_q;  // varlen: rows of the packed q / o (cu_seqlens_q is clamped to it)
  size_t ws_o_offset;
};
cudaError_t launch_merge(const MergeArgs& a, cudaStream_t stream);

// ---- tcgen05 prefill (bf16, d in {64, 128, 256}) ----
struct TcFwdArgs {
  CUtensorMap tm_q, tm_k, tm_v;  // 3-D maps, box {64, 1 or 128 (d = 256 K/V: 64), ...}, 128-byte swizzle
  uint16_t* o;
  float* lse;
  const int32_t* cu_q;  // varlen (packed) mode if non-null
  const int32_t* cu_k;
  int B, Hq, Hkv, Nq, Nk, d, causal;  // packed mode: Nq, Nk = total rows of q and k
  int num_seqs;
  int small_rows_limit;  // varlen: sequences with n_q * g <= this are skipped here
  int max_pairs;         // work items per (sequence, head): pairs of 128-row query tiles (d = 256: tiles)
  int window;            // > 0: sliding window of that many keys ending at the causal limit
  int band_units;        // (sequence, head) units per band of the item list (at least 1)
  int head_pair;         // d = 128, even g: a work item is one query tile of two heads that share
                         // a KV head (units are head pairs, max_pairs counts query tiles)
  float scale_log2;
  uint64_t timeout_ns;
};
// `sched`: two zeroed device counters (next item, CTAs finished) owned by this launch alone;
// the kernel leaves them zeroed again when it completes.
cudaError_t launch_prefill_tc(const TcFwdArgs& a, unsigned int* status, unsigned int* sched, cudaStream_t stream);
// Head dim 256: one 128-row query tile per item, 64-key K/V tiles (the K/V maps' box is 64 rows
// or tokens high), a.max_pairs = query tiles per (sequence, head).
cudaError_t launch_prefill_tc256(const TcFwdArgs& a, unsigned int* status, unsigned int* sched, cudaStream_t stream);

// ---- attention of drafted token trees over a cache ----
// A tile is kTreeRows rows, a row being one (node, query head) pair of the KV head's group; a tile
// holds kTreeRows / g whole nodes, a unit one or two tiles (tree_row_tiles) of one KV head.
constexpr int kTreeMaxNodes = 1024;  // drafted nodes a sequence
constexpr int kTreeRows = 128;
constexpr int kTreeMaxCtas = 304;    // persistent CTAs, two per SM (tree_max_ctas)
constexpr int kTreeMergeBytes = 12288;
// Tiles' time that a unit takes beside its tiles (its own Q, drafts, output; a tile is half the bytes at
// d = 64). 48 ragged requests at d = 64: 82.7 us at 3 and 4, 86.3 at 6 (before the hot loops were taken apart
// 118 at 0); 30 ragged requests of two row tiles at d = 128: 82.6 us at 1, 78.0 at 2, 80.7 at 3. At d = 256 it
// matters little: at 1, 2, 4 and 6, 4 ragged requests up to 12000 keys took 40.1, 39.7, 39.4 and 40.0 us, 30 up
// to 6000 over pages 74.2, 74.8, 75.7 and 76.8, 64 of 700 keys 30.6, 29.2, 29.8 and 30.6.
__host__ __device__ constexpr int tree_unit_cost(int d) { return d == 64 ? 4 : 2; }
// What the merge has to do at the boundary between a CTA and the one before it (of its KV head: head_group
// CTAs before), written by the later: something if that is the first boundary inside a unit.
struct TreeMergeRec {
  int rows0, rows1;      // rows of the unit's row tiles (rows0 0: nothing to merge)
  int node0, node_step;  // packed row of the tiles' first node: node0 + w node_step
  int hkv;
  int slot0;             // the CTA before has its part in this slot, the later ones in slot 0
  int last;              // the last CTA with a part
  int pad;
};
static_assert(sizeof(TreeMergeRec) == 32 && kTreeMaxCtas * sizeof(TreeMergeRec) <= kTreeMergeBytes, "merge records");
struct TreeArgs {
  CUtensorMap tm_q;        // {d, Hq, total_q}, box {64, g, tile_rows / g}
  CUtensorMap tm_k, tm_v;  // contiguous {d, cap, B * Hkv}, box {64, tile keys, 1}; paged {d, Hkv, pool rows},
                           // box {64, 1, piece}
  CUtensorMap tm_kn, tm_vn;  // {d, Hkv, total_q}, box {64, 1, new_box}
  const uint16_t* q;      // bf16 bits; node t of the packed batch at q + t * q_stride, heads d apart
  const uint16_t* k;      // cache: contiguous [B, Hkv, cap, d] or pages [num_pages, page_size, Hkv, d]
  const uint16_t* v;
  const uint16_t* k_new;  // drafted rows, node t at k_new + t * k_new_stride, KV heads d apart
  const uint16_t* v_new;
  uint16_t* o;            // [total_q, Hq, d]
  float* lse;             // [total_q, Hq] or null
  const int32_t* nk;      // [num_seqs] context keys (clamped to kv_cap)
  const int32_t* cu_q;    // [num_seqs + 1] (clamped to total_q)
  const uint64_t* mask;   // [total_q, mask_words]: bit j = draft j of the node's own sequence is seen
  const int32_t* block_table;  // paged cache when non-null: [num_seqs, max_pages]
  int64_t q_stride, k_new_stride, v_new_stride;
  TreeMergeRec* merge;    // workspace: [ctas]
  float* partial;         // workspace: [ctas][2][row tiles][kTreeRows * (d + 2)]
  int num_seqs, total_q, max_nodes, mask_words;
  int Hq, Hkv, g, d;
  int kv_cap;             // keys a sequence's cache can hold
  int page_size, max_pages, num_pages;
  int tile_rows, tile_nodes;  // tree_tile_rows(max_nodes, g, d); / g
  int piece;              // paged: rows of a copy, a power of two that divides page_size
  int new_box;            // rows of a copy of drafted rows
  int head_group, head_groups;  // KV heads that a group of CTAs takes side by side; Hkv / head_group
  int groups;             // groups of CTAs of the attention kernel
  int merges, merge_warps;  // units that may have to be merged; warps that share out one's parts
  float scale_log2;
  unsigned int* status;
  uint64_t timeout_ns;
};
// Row tiles of a unit: two (d <= 128) when a sequence may fill more than one, so that the K and V
// tiles of a unit serve twice the rows.
inline int tree_row_tiles(int max_nodes, int g, int d) { return d <= 128 && max_nodes > kTreeRows / g ? 2 : 1; }
inline int tree_max_ctas(int row_tiles, int d) { return row_tiles == 1 && d <= 128 ? kTreeMaxCtas : kTreeMaxCtas / 2; }
// Rows of a tile that hold nodes: 64 where no sequence has more (d <= 128).
inline int tree_tile_rows(int max_nodes, int g, int d) {
  return d <= 128 && static_cast<int64_t>(max_nodes) * g <= 64 ? 64 : kTreeRows;
}
inline size_t tree_ws_bytes(int max_nodes, int g, int d) {
  const int tiles = tree_row_tiles(max_nodes, g, d);
  return kTreeMergeBytes +
         static_cast<size_t>(tree_max_ctas(tiles, d)) * 2 * tiles * kTreeRows * (d + 2) * sizeof(float);
}
// The most units, and places (tree_unit_cost and the key tiles of every unit), that the lengths of a call may
// make (places are int in the kernel: the host refuses more).
inline int64_t tree_most_units(const TreeArgs& a) {
  const int unit_nodes = tree_row_tiles(a.max_nodes, a.g, a.d) * (tree_tile_rows(a.max_nodes, a.g, a.d) / a.g);
  const int64_t seqs = a.num_seqs < a.total_q ? a.num_seqs : a.total_q;
  return a.Hkv * (seqs + a.total_q / unit_nodes);
}
inline int64_t tree_most_tiles(const TreeArgs& a) {
  const int keys = a.d == 256 ? 64 : 128;
  return tree_most_units(a) *
         ((static_cast<int64_t>(a.kv_cap) + keys - 1) / keys + (a.max_nodes + keys - 1) / keys + tree_unit_cost(a.d));
}
// Fills the maps and sizes that follow from the others, launches the attention and the merge.
cudaError_t launch_tree(TreeArgs& a, void* workspace, cudaStream_t stream);

#ifdef __CUDACC__
// Launches a kernel whose threads all pass griddepcontrol.wait before they touch memory: it may be set up
// while the kernel before it in the stream ends.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}
#endif

// ---- paged cache bookkeeping ----
struct TreeMaskArgs {
  const int32_t* parents;
  const int32_t* cu_q;
  const int32_t* nk;  // or null
  uint64_t* mask;
  int32_t* positions;  // or null
  int num_seqs, total_q, max_nodes, words;
};
cudaError_t launch_tree_mask(const TreeMaskArgs& a, cudaStream_t stream);

struct PlanArgs {
  const int32_t* nk;
  const int32_t* n_new;
  int32_t* table;
  const int32_t* held;
  const int32_t* free_pages;
  const int32_t* free_count;
  int32_t* nk_out;
  int32_t* held_out;
  int32_t* cu;
  int32_t* slots;
  int32_t* free_out;
  int B, page_size, max_pages, free_cap, num_tokens;
};
cudaError_t launch_kv_plan(const PlanArgs& a, cudaStream_t stream);

struct AppendArgs {
  const uint16_t* k_new;
  const uint16_t* v_new;
  const int32_t* slots;
  const int32_t* rows;  // or null: slot i takes row i
  void* k_pages;
  void* v_pages;
  const float* k_scale;  // non-null: E4M3 pages
  const float* v_scale;
  int64_t k_stride, v_stride;  // elements between rows of k_new / v_new
  int num_slots, num_rows;     // num_rows: rows of k_new and v_new
  int64_t pool_rows;           // num_pages * page_size
  int row_elems;               // Hkv * d
};
cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t stream);

// Timeout self-test: one CTA waits on a barrier that is never arrived at.
cudaError_t launch_wait_timeout_probe(uint64_t timeout_ns, unsigned int* status, cudaStream_t stream);

// Bookkeeping shared by every entry point (defined in api.cu): record a failed CUDA call for
// bwattn_last_cuda_error(), count a successful launch for bwattn_launch_count().
void record_cuda_error(cudaError_t e);
void count_launch();
// `n` zeroed merge tickets on the current device for one launch of the split-K kernel (null
// when the request exceeds the ticket pool: the caller then launches the merge kernel).
cudaError_t merge_tickets(int n, unsigned int** out);
// 3-D bf16 tensor map {d, dim1, dim2} with strides in elements, box {64, box1, box2}, 128-byte
// swizzle, zero fill out of bounds.
cudaError_t make_map_bf16(CUtensorMap* m, const void* base, int d, int64_t dim1, int64_t dim2, int64_t stride1_elems,
                          int64_t stride2_elems, int box1, int box2);
// The device status word of the current device and the bound on a kernel's waits.
cudaError_t status_word(unsigned int** out);
uint64_t wait_timeout_ns();

// Float offset of the o[] block of the split-K workspace (after the (m, l) pairs, 256-byte aligned).
inline size_t splitk_o_offset(int units, int num_splits, int rows_max) {
  return (static_cast<size_t>(units) * num_splits * rows_max * 2 + 63) & ~static_cast<size_t>(63);
}
inline size_t splitk_ws_bytes(int units, int num_splits, int rows_max, int d) {
  return (splitk_o_offset(units, num_splits, rows_max) + static_cast<size_t>(units) * num_splits * rows_max * d) *
         sizeof(float);
}

}  // namespace bw
