// C-ABI of the entry points around a paged cache's attention (norm and rotation of q and k, chunks over the
// pages, verification of drafted trees): argument validation and dispatch. See include/bwattn.h for the contracts.
#include <math.h>
#include <stdint.h>

#include "../../include/bwattn.h"
#include "checks.h"
#include "kernels.h"

namespace {

// what attn_chunk_paged takes, and the size of its workspace is given for: sizes in range (else INVALID_ARG) ...
bool chunk_range(int num_seqs, int max_seqlen_q, int Hq, int Hkv, int d) {
  return num_seqs >= 0 && num_seqs <= 65535 && max_seqlen_q >= 0 && Hq > 0 && Hq <= 65535 && Hkv > 0 && d > 0 && Hq % Hkv == 0;
}
// ... that the kernels implement (else UNSUPPORTED)
bool chunk_supported(int g, int d) { return head_dim(d) && g <= bw::kTreeRows; }

}  // namespace

extern "C" {

size_t attn_chunk_workspace_size(int num_seqs, int max_seqlen_q, int Hq, int Hkv, int d) {
  if (!chunk_range(num_seqs, max_seqlen_q, Hq, Hkv, d) || !chunk_supported(Hq / Hkv, d) || num_seqs == 0 || max_seqlen_q == 0)
    return 0;
  return bw::tree_ws_bytes(max_seqlen_q, Hq / Hkv, d);
}

int attn_chunk_paged(const void* q, const void* k_pages, const void* v_pages, const int32_t* block_table, void* o, float* lse,
                     const int32_t* nk, const int32_t* cu_seqlens_q, int num_seqs, int total_q, int max_seqlen_q,
                     int page_size, int num_pages, int max_pages_per_seq, int Hq, int Hkv, int d, int64_t q_stride, int causal,
                     float scale, void* workspace, size_t workspace_bytes, void* stream) {
  if (!chunk_range(num_seqs, max_seqlen_q, Hq, Hkv, d) || total_q < 0 || !(isfinite(scale) && scale > 0.f) ||
      (causal != 0 && causal != 1) || !page_sizes(page_size, num_pages) || max_pages_per_seq <= 0 ||
      static_cast<int64_t>(max_pages_per_seq) * page_size > 0x7fffffff)
    return BWATTN_ERR_INVALID_ARG;
  const int g = Hq / Hkv;
  if (!chunk_supported(g, d)) return BWATTN_ERR_UNSUPPORTED;
  if (num_seqs == 0 || total_q == 0 || max_seqlen_q == 0) return BWATTN_OK;
  if (!good(q, 16) || !good(k_pages, 16) || !good(v_pages, 16) || !good(block_table, 4) || !good(o, 16) ||
      !good_or_null(lse, 4) || !good(nk, 4) || !good(cu_seqlens_q, 4) || !good(workspace, 16))
    return BWATTN_ERR_INVALID_ARG;
  if (!row_stride(q_stride, static_cast<int64_t>(Hq) * d)) return BWATTN_ERR_INVALID_ARG;
  if (workspace_bytes < bw::tree_ws_bytes(max_seqlen_q, g, d)) return BWATTN_ERR_INVALID_ARG;
  bw::TreeArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k_pages);
  a.v = static_cast<const uint16_t*>(v_pages);
  a.o = static_cast<uint16_t*>(o);
  a.lse = lse;
  a.nk = nk;
  a.cu_q = cu_seqlens_q;
  a.block_table = block_table;
  a.q_stride = q_stride;
  a.num_seqs = num_seqs;
  a.total_q = total_q;
  a.max_nodes = max_seqlen_q < total_q ? max_seqlen_q : total_q;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.g = g;
  a.d = d;
  a.kv_cap = max_pages_per_seq * page_size;
  a.page_size = page_size;
  a.max_pages = max_pages_per_seq;
  a.num_pages = num_pages;
  a.causal = causal;
  a.scale_log2 = scale * bw::kLog2e;
  // a tile takes up to 4 places of the list, which the heads of a group share
  if (4 * bw::tree_most_tiles(a) / bw::tree_head_group(Hkv, 8) > 0x7fffffff || static_cast<int64_t>(a.kv_cap) + a.max_nodes > 0x7fffffff)
    return BWATTN_ERR_UNSUPPORTED;
  return done(bw::launch_tree(a, workspace, static_cast<cudaStream_t>(stream)));
}

int attn_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out, const int32_t* positions, const int32_t* axes,
                      const float* inv_freq, const void* q_weight, const void* k_weight, float eps, int num_rows,
                      int num_axes, int pairs, int interleaved, int Hq, int Hkv, int d, int64_t q_stride, int64_t k_stride,
                      int64_t q_out_stride, int64_t k_out_stride, void* stream) {
  if (num_rows < 0 || num_axes < 1 || pairs < 0 || Hq <= 0 || Hq > 65535 || Hkv <= 0 || Hkv > 65535 || d <= 0 ||
      (interleaved != 0 && interleaved != 1) || !(isfinite(eps) && eps >= 0.f))
    return BWATTN_ERR_INVALID_ARG;
  if (!head_dim(d)) return BWATTN_ERR_UNSUPPORTED;
  if (pairs > d / 2) return BWATTN_ERR_INVALID_ARG;
  if (num_rows == 0) return BWATTN_OK;
  if (!good(q, 16) || !good(k, 16) || !good(q_out, 16) || !good(k_out, 16) || !good_or_null(q_weight, 16) ||
      !good_or_null(k_weight, 16) || !good_or_null(axes, 4) || !good_or_null(positions, 4) || !good_or_null(inv_freq, 4) ||
      (pairs > 0 && (!positions || !inv_freq)))
    return BWATTN_ERR_INVALID_ARG;
  const int64_t qw = static_cast<int64_t>(Hq) * d, kw = static_cast<int64_t>(Hkv) * d;
  if (!row_stride(q_stride, qw) || !row_stride(k_stride, kw) || !row_stride(q_out_stride, qw) || !row_stride(k_out_stride, kw))
    return BWATTN_ERR_INVALID_ARG;
  // in place: a row is written where it was read
  if ((q == q_out && q_stride != q_out_stride) || (k == k_out && k_stride != k_out_stride) || q == k_out || k == q_out || q_out == k_out)
    return BWATTN_ERR_INVALID_ARG;
  bw::RopeArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.k_out = static_cast<uint16_t*>(k_out);
  a.positions = positions;
  a.axes = axes;
  a.freq = inv_freq;
  a.q_weight = static_cast<const uint16_t*>(q_weight);
  a.k_weight = static_cast<const uint16_t*>(k_weight);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.q_out_stride = q_out_stride;
  a.k_out_stride = k_out_stride;
  a.num_rows = num_rows;
  a.num_axes = num_axes;
  a.pairs = pairs;
  a.interleaved = interleaved;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.eps = eps;
  const cudaError_t e = bw::launch_qk_rope(a, static_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) bw::count_launch();
  return done(e);
}

int attn_tree_verify(const int32_t* tokens, const int32_t* parents, const int32_t* cu_seqlens_q, const float* target_probs,
                     const float* draft_probs, const float* uniforms, const float* sample_uniforms, int32_t* accepted,
                     int32_t* counts, int32_t* next_tokens, int num_seqs, int total_q, int max_nodes, int vocab,
                     int64_t target_stride, int64_t draft_stride, void* stream) {
  if (num_seqs < 0 || num_seqs > 65535 || total_q < 0 || max_nodes < 0 || vocab < 1) return BWATTN_ERR_INVALID_ARG;
  if (max_nodes > bw::kTreeMaxNodes || vocab > bw::kVerifyMaxVocab) return BWATTN_ERR_UNSUPPORTED;
  if (num_seqs == 0 && total_q == 0) return BWATTN_OK;
  if (num_seqs > 0 && (!good(cu_seqlens_q, 4) || !good(sample_uniforms, 4) || !good(counts, 4) || !good(next_tokens, 4)))
    return BWATTN_ERR_INVALID_ARG;
  if (total_q > 0 && (!good(tokens, 4) || !good(parents, 4) || !good(target_probs, 4) || !good_or_null(draft_probs, 4) ||
                      !good(uniforms, 4) || !good(accepted, 4)))
    return BWATTN_ERR_INVALID_ARG;
  const int64_t most = static_cast<int64_t>(1) << 38;
  if (target_stride < vocab || target_stride >= most || (draft_probs && (draft_stride < vocab || draft_stride >= most)))
    return BWATTN_ERR_INVALID_ARG;
  // every CTA of a request reads all of its inputs, so no output may stand in an input's place, nor in another output's
  const void* in[] = {tokens, parents, cu_seqlens_q, target_probs, draft_probs, uniforms, sample_uniforms};
  const void* out[] = {accepted, counts, next_tokens};
  for (const void* y : out)
    for (const void* x : in)
      if (x && x == y) return BWATTN_ERR_INVALID_ARG;
  if (accepted == counts || accepted == next_tokens || (counts && counts == next_tokens)) return BWATTN_ERR_INVALID_ARG;
  bw::VerifyArgs a{tokens, parents, cu_seqlens_q, target_probs, draft_probs, uniforms, sample_uniforms, accepted, counts,
                   next_tokens, target_stride, draft_stride, num_seqs, total_q, max_nodes, vocab, nullptr, 0};
  const cudaError_t e = bw::launch_tree_verify(a, static_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) bw::count_launch();
  return done(e);
}

}  // extern "C"
