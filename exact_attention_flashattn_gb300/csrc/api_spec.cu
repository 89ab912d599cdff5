// C-ABI of the speculative-decoding entry points (tree attention, tree masks, paged plans and
// appends): argument validation and dispatch. See include/bwattn.h for the contracts.
#include <math.h>
#include <stdint.h>

#include "../../include/bwattn.h"
#include "checks.h"
#include "kernels.h"

namespace {

// what the tree calls take, and the size of their workspace is given for: sizes in range (else INVALID_ARG) ...
bool tree_range(int num_seqs, int max_nodes, int Hq, int Hkv, int d) {
  return num_seqs >= 0 && num_seqs <= 65535 && max_nodes >= 0 && Hq > 0 && Hq <= 65535 && Hkv > 0 && d > 0 && Hq % Hkv == 0;
}
// ... that the kernels implement (else UNSUPPORTED)
bool tree_supported(int max_nodes, int g, int d) { return head_dim(d) && g <= bw::kTreeRows && max_nodes <= bw::kTreeMaxNodes; }

int tree_impl(const void* q, const void* k, const void* v, const void* k_new, const void* v_new, void* o, float* lse,
              const int32_t* nk, const int32_t* cu_seqlens_q, const uint64_t* mask, const int32_t* block_table,
              int num_seqs, int total_q, int max_nodes, int kv_cap, int page_size, int num_pages, int max_pages,
              int Hq, int Hkv, int d, int64_t q_stride, int64_t k_new_stride, int64_t v_new_stride, float scale,
              void* workspace, size_t workspace_bytes, void* stream) {
  if (!tree_range(num_seqs, max_nodes, Hq, Hkv, d) || total_q < 0 || kv_cap < 0 || !(isfinite(scale) && scale > 0.f))
    return BWATTN_ERR_INVALID_ARG;
  const int g = Hq / Hkv;
  if (!tree_supported(max_nodes, g, d)) return BWATTN_ERR_UNSUPPORTED;
  if (num_seqs == 0 || total_q == 0 || max_nodes == 0) return BWATTN_OK;
  if (!good(q, 16) || !good(k_new, 16) || !good(v_new, 16) || !good(o, 16) || !good_or_null(lse, 4) || !good(nk, 4) ||
      !good(cu_seqlens_q, 4) || !good(mask, 8) || !good(workspace, 16))
    return BWATTN_ERR_INVALID_ARG;
  if (kv_cap > 0 && (!good(k, 16) || !good(v, 16))) return BWATTN_ERR_INVALID_ARG;
  if (!row_stride(q_stride, static_cast<int64_t>(Hq) * d) || !row_stride(k_new_stride, static_cast<int64_t>(Hkv) * d) ||
      !row_stride(v_new_stride, static_cast<int64_t>(Hkv) * d))
    return BWATTN_ERR_INVALID_ARG;
  if (workspace_bytes < bw::tree_ws_bytes(max_nodes, g, d)) return BWATTN_ERR_INVALID_ARG;
  bw::TreeArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.k_new = static_cast<const uint16_t*>(k_new);
  a.v_new = static_cast<const uint16_t*>(v_new);
  a.o = static_cast<uint16_t*>(o);
  a.lse = lse;
  a.nk = nk;
  a.cu_q = cu_seqlens_q;
  a.mask = mask;
  a.block_table = block_table;
  a.q_stride = q_stride;
  a.k_new_stride = k_new_stride;
  a.v_new_stride = v_new_stride;
  a.num_seqs = num_seqs;
  a.total_q = total_q;
  a.max_nodes = max_nodes;
  a.mask_words = (max_nodes + 63) / 64;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.g = g;
  a.d = d;
  a.kv_cap = kv_cap;
  a.page_size = page_size;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.scale_log2 = scale * bw::kLog2e;
  if (bw::tree_most_tiles(a) > 0x7fffffff) return BWATTN_ERR_UNSUPPORTED;
  return done(bw::launch_tree(a, workspace, static_cast<cudaStream_t>(stream)));
}

int append_impl(const void* k_new, const void* v_new, const int32_t* slots, const int32_t* rows, void* k_pages,
                void* v_pages, const float* k_scale, const float* v_scale, bool fp8, int num_slots, int num_rows,
                int page_size, int num_pages, int Hkv, int d, int64_t k_new_stride, int64_t v_new_stride,
                void* stream) {
  if (num_slots < 0 || num_rows < 0 || Hkv <= 0 || d <= 0 || Hkv > 65535 || !page_sizes(page_size, num_pages))
    return BWATTN_ERR_INVALID_ARG;
  if (!head_dim(d)) return BWATTN_ERR_UNSUPPORTED;
  if (num_slots == 0 || num_rows == 0) return BWATTN_OK;
  if (!rows && num_slots > num_rows) return BWATTN_ERR_INVALID_ARG;
  if (!good(k_new, 16) || !good(v_new, 16) || !good(slots, 4) || !good_or_null(rows, 4) || !good(k_pages, 16) ||
      !good(v_pages, 16) || (fp8 && (!good(k_scale, 16) || !good(v_scale, 16))))
    return BWATTN_ERR_INVALID_ARG;
  if (!row_stride(k_new_stride, static_cast<int64_t>(Hkv) * d) || !row_stride(v_new_stride, static_cast<int64_t>(Hkv) * d))
    return BWATTN_ERR_INVALID_ARG;
  bw::AppendArgs a{};
  a.k_new = static_cast<const uint16_t*>(k_new);
  a.v_new = static_cast<const uint16_t*>(v_new);
  a.slots = slots;
  a.rows = rows;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.k_scale = fp8 ? k_scale : nullptr;
  a.v_scale = fp8 ? v_scale : nullptr;
  a.k_stride = k_new_stride;
  a.v_stride = v_new_stride;
  a.num_slots = num_slots;
  a.num_rows = num_rows;
  a.pool_rows = static_cast<int64_t>(num_pages) * page_size;
  a.row_elems = Hkv * d;
  cudaError_t e = bw::launch_kv_append(a, static_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) bw::count_launch();
  return done(e);
}

}  // namespace

extern "C" {

size_t attn_tree_workspace_size(int num_seqs, int max_nodes, int Hq, int Hkv, int d) {
  if (!tree_range(num_seqs, max_nodes, Hq, Hkv, d) || !tree_supported(max_nodes, Hq / Hkv, d) || num_seqs == 0 || max_nodes == 0)
    return 0;
  return bw::tree_ws_bytes(max_nodes, Hq / Hkv, d);
}

int attn_tree(const void* q, const void* kcache, const void* vcache, const void* k_new, const void* v_new, void* o,
              float* lse, const int32_t* nk, const int32_t* cu_seqlens_q, const uint64_t* mask, int num_seqs,
              int total_q, int max_nodes, int nk_cap, int Hq, int Hkv, int d, int64_t q_stride, int64_t k_new_stride,
              int64_t v_new_stride, float scale, void* workspace, size_t workspace_bytes, void* stream) {
  return tree_impl(q, kcache, vcache, k_new, v_new, o, lse, nk, cu_seqlens_q, mask, nullptr, num_seqs, total_q,
                   max_nodes, nk_cap, 0, 0, 0, Hq, Hkv, d, q_stride, k_new_stride, v_new_stride, scale, workspace,
                   workspace_bytes, stream);
}

int attn_tree_paged(const void* q, const void* k_pages, const void* v_pages, const int32_t* block_table,
                    const void* k_new, const void* v_new, void* o, float* lse, const int32_t* nk,
                    const int32_t* cu_seqlens_q, const uint64_t* mask, int num_seqs, int total_q, int max_nodes,
                    int page_size, int num_pages, int max_pages_per_seq, int Hq, int Hkv, int d, int64_t q_stride,
                    int64_t k_new_stride, int64_t v_new_stride, float scale, void* workspace, size_t workspace_bytes,
                    void* stream) {
  if (!page_sizes(page_size, num_pages) || max_pages_per_seq <= 0 ||
      static_cast<int64_t>(max_pages_per_seq) * page_size > 0x7fffffff)
    return BWATTN_ERR_INVALID_ARG;
  if (num_seqs > 0 && total_q > 0 && max_nodes > 0 && !good(block_table, 4)) return BWATTN_ERR_INVALID_ARG;
  return tree_impl(q, k_pages, v_pages, k_new, v_new, o, lse, nk, cu_seqlens_q, mask, block_table, num_seqs, total_q,
                   max_nodes, max_pages_per_seq * page_size, page_size, num_pages, max_pages_per_seq, Hq, Hkv, d,
                   q_stride, k_new_stride, v_new_stride, scale, workspace, workspace_bytes, stream);
}

int attn_tree_mask(const int32_t* parents, const int32_t* cu_seqlens_q, const int32_t* nk, uint64_t* mask,
              int32_t* positions, int num_seqs, int total_q, int max_nodes, void* stream) {
  if (num_seqs < 0 || total_q < 0 || max_nodes < 0) return BWATTN_ERR_INVALID_ARG;
  if (max_nodes > bw::kTreeMaxNodes) return BWATTN_ERR_UNSUPPORTED;
  if (num_seqs == 0 || total_q == 0 || max_nodes == 0) return BWATTN_OK;
  if (!good(parents, 4) || !good(cu_seqlens_q, 4) || !good_or_null(nk, 4) || !good(mask, 8) ||
      !good_or_null(positions, 4))
    return BWATTN_ERR_INVALID_ARG;
  const bw::TreeMaskArgs a{parents, cu_seqlens_q, nk, mask, positions, num_seqs, total_q, max_nodes, (max_nodes + 63) / 64};
  cudaError_t e = bw::launch_tree_mask(a, static_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) bw::count_launch();
  return done(e);
}

int kv_plan_paged(const int32_t* nk, const int32_t* n_new, int32_t* block_table, const int32_t* held,
                  const int32_t* free_pages, const int32_t* free_count, int32_t* nk_out, int32_t* held_out,
                  int32_t* cu_seqlens, int32_t* slots, int32_t* free_count_out, int B, int page_size,
                  int max_pages_per_seq, int free_capacity, int num_tokens, void* stream) {
  if (B < 0 || num_tokens < 0 || free_capacity < 0 || max_pages_per_seq <= 0 || !page_sizes(page_size, 1) ||
      static_cast<int64_t>(max_pages_per_seq) * page_size > 0x7fffffff ||
      static_cast<int64_t>(B) * max_pages_per_seq > 0x7fffffff)
    return BWATTN_ERR_INVALID_ARG;
  if (!good(free_count, 4) || !good(free_count_out, 4) || !good(cu_seqlens, 4) || !good_or_null(free_pages, 4) ||
      (free_capacity > 0 && !free_pages) || !good_or_null(slots, 4) || (num_tokens > 0 && !slots))
    return BWATTN_ERR_INVALID_ARG;
  if (B > 0 && (!good(nk, 4) || !good(n_new, 4) || !good(block_table, 4) || !good(held, 4) || !good(nk_out, 4) ||
                !good(held_out, 4)))
    return BWATTN_ERR_INVALID_ARG;
  // every CTA reads all of the inputs, so no output may stand in an input's place
  const void* in[] = {nk, n_new, held, free_pages, free_count};
  const void* out[] = {block_table, nk_out, held_out, cu_seqlens, slots, free_count_out};
  for (const void* x : in)
    for (const void* y : out)
      if (x && x == y) return BWATTN_ERR_INVALID_ARG;
  const bw::PlanArgs a{nk,     n_new,      block_table, held,           free_pages, free_count,
                       nk_out, held_out,   cu_seqlens,  slots,          free_count_out, B,
                       page_size, max_pages_per_seq, free_capacity, num_tokens};
  cudaError_t e = bw::launch_kv_plan(a, static_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) bw::count_launch();
  return done(e);
}

int kv_append_paged(const void* k_new, const void* v_new, const int32_t* slots, const int32_t* rows, void* k_pages,
                    void* v_pages, int num_slots, int num_rows, int page_size, int num_pages, int Hkv, int d,
                    int64_t k_new_stride, int64_t v_new_stride, void* stream) {
  return append_impl(k_new, v_new, slots, rows, k_pages, v_pages, nullptr, nullptr, false, num_slots, num_rows,
                     page_size, num_pages, Hkv, d, k_new_stride, v_new_stride, stream);
}

int kv_append_paged_fp8(const void* k_new, const void* v_new, const int32_t* slots, const int32_t* rows,
                        void* k_pages, void* v_pages, const float* k_scale, const float* v_scale, int num_slots,
                        int num_rows, int page_size, int num_pages, int Hkv, int d, int64_t k_new_stride,
                        int64_t v_new_stride, void* stream) {
  return append_impl(k_new, v_new, slots, rows, k_pages, v_pages, k_scale, v_scale, true, num_slots, num_rows,
                     page_size, num_pages, Hkv, d, k_new_stride, v_new_stride, stream);
}

}  // extern "C"
