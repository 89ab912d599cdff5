// Paged KV cache bookkeeping on the GPU: ancestor masks of drafted token trees, block tables and
// slot maps from request lengths, and K/V rows written into the pages (bf16 or E4M3 codes).
#include "kernels.h"
#include "ptx.cuh"

namespace bw {

namespace {

// ---------------------------------------------------------------- tree masks
//
// mask[i] = mask[parent(i)] | bit i, position[i] = nk + depth(i). A parent precedes its children
// (anything else counts as a root), so a walk from node i up its parents visits falling indices and
// ends. One CTA per sequence holds the parents in shared memory; a thread makes one 64-bit word of
// one node's mask: it walks from the node until the indices fall below its word, and the thread of
// word 0, which walks to the root, counts the depth.
constexpr int kMaskThreads = 256;
constexpr int kMaskMaxNodes = 1024;

__global__ void __launch_bounds__(kMaskThreads) tree_mask_kernel(const TreeMaskArgs a) {
  __shared__ int16_t parent[kMaskMaxNodes];
  const int seq = blockIdx.x;
  const int t0 = min(max(a.cu_q[seq], 0), a.total_q);
  const int n = min(min(max(a.cu_q[seq + 1] - t0, 0), a.total_q - t0), a.max_nodes);
  for (int i = threadIdx.x; i < n; i += kMaskThreads) {
    const int p = a.parents[t0 + i];
    parent[i] = static_cast<int16_t>(p >= 0 && p < i ? p : -1);
  }
  __syncthreads();
  const int base = a.nk ? a.nk[seq] : 0;
  for (int it = threadIdx.x; it < n * a.words; it += kMaskThreads) {
    const int i = it / a.words, w = it % a.words;
    uint64_t bits = 0;
    int depth = -1;
    for (int j = i; j >= 64 * w; j = parent[j]) {
      if ((j >> 6) == w) bits |= 1ull << (j & 63);
      ++depth;
    }
    a.mask[static_cast<int64_t>(t0 + i) * a.words + w] = bits;
    if (w == 0 && a.positions) a.positions[t0 + i] = base + depth;
  }
}

// ---------------------------------------------------------------- block tables and slot maps
//
// need_b = max(0, min(ceil((nk_b + new_b) / P), max_pages) - held_b) pages are taken from the top of
// the free stack, request after request: page k >= held_b of request b is
// free[count - 1 - (first_b + k - held_b)], first_b the sum of the needs before b. Every CTA scans
// all requests, kPlanThreads at a time (two prefix sums, 64-bit: lengths come from the device and
// their sum may pass 32 bits), and writes its share of the tokens' slots, of the new table entries
// and of the per-request outputs, so no CTA waits for another: a token's page is worked out from
// the old table or the free stack, never read from what this launch writes.
constexpr int kPlanThreads = 512;

__device__ __forceinline__ int plan_page(const PlanArgs& a, int count, int64_t i) {
  return i < count ? a.free_pages[count - 1 - i] : -1;  // past the stack: no page
}

__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(const PlanArgs a) {
  constexpr int kW = kPlanThreads / 32;
  __shared__ int64_t s_tok[kPlanThreads + 1], s_page[kPlanThreads + 1];  // exclusive sums of the chunk
  __shared__ int s_nk[kPlanThreads], s_held[kPlanThreads];
  __shared__ int64_t s_wt[kW], s_wp[kW];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int count = min(max(*a.free_count, 0), a.free_cap);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kPlanThreads;
  const int64_t me = static_cast<int64_t>(blockIdx.x) * kPlanThreads + tid;
  int64_t tok_sum = 0, page_sum = 0;
  for (int b0 = 0, chunk = 0; b0 < a.B; b0 += kPlanThreads, ++chunk) {
    const int b = b0 + tid;
    int nk = 0, held = 0;
    int64_t add = 0, need = 0;
    if (b < a.B) {
      nk = max(a.nk[b], 0);
      held = min(max(a.held[b], 0), a.max_pages);
      add = max(a.n_new[b], 0);
      const int64_t want = min((nk + add + a.page_size - 1) / a.page_size, static_cast<int64_t>(a.max_pages));
      need = max(want - held, static_cast<int64_t>(0));
    }
    int64_t st = add, sp = need;  // inclusive sums over the warp, then the block
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, st, off), y = __shfl_up_sync(0xffffffffu, sp, off);
      if (lane >= off) {
        st += x;
        sp += y;
      }
    }
    if (lane == 31) {
      s_wt[warp] = st;
      s_wp[warp] = sp;
    }
    __syncthreads();
    int64_t ct = 0, cp = 0;  // chunk totals; the warps before this one
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      if (w == warp) {
        st += ct;
        sp += cp;
      }
      ct += s_wt[w];
      cp += s_wp[w];
    }
    s_tok[tid] = tok_sum + st - add;
    s_page[tid] = page_sum + sp - need;
    s_nk[tid] = nk;
    s_held[tid] = held;
    if (b < a.B && chunk % gridDim.x == blockIdx.x) {
      a.nk_out[b] = static_cast<int>(min(nk + add, static_cast<int64_t>(0x7fffffff)));
      a.held_out[b] = held + static_cast<int>(need);
      a.cu[b] = static_cast<int>(min(tok_sum + st - add, static_cast<int64_t>(0x7fffffff)));
    }
    if (tid == 0) {
      s_tok[kPlanThreads] = tok_sum + ct;
      s_page[kPlanThreads] = page_sum + cp;
    }
    __syncthreads();
    // the request of an item: the last one whose exclusive sum is at most the item's index
    auto request = [&](const int64_t* sums, int64_t x) {
      int lo = 0;
#pragma unroll
      for (int w = kPlanThreads / 2; w > 0; w >>= 1)
        if (sums[lo + w] <= x) lo += w;
      return lo;
    };
    for (int64_t x = page_sum + me; x < page_sum + cp; x += step) {
      const int r = request(s_page, x);
      const int64_t k = s_held[r] + (x - s_page[r]);
      a.table[static_cast<int64_t>(b0 + r) * a.max_pages + k] = plan_page(a, count, x);
    }
    for (int64_t x = tok_sum + me; x < min(tok_sum + ct, static_cast<int64_t>(a.num_tokens)); x += step) {
      const int r = request(s_tok, x);
      const int64_t pos = s_nk[r] + (x - s_tok[r]);
      const int64_t k = pos / a.page_size;
      int64_t slot = -1;
      if (k < a.max_pages) {
        const int page = k < s_held[r] ? a.table[static_cast<int64_t>(b0 + r) * a.max_pages + k]
                                       : plan_page(a, count, s_page[r] + (k - s_held[r]));
        if (page >= 0) slot = static_cast<int64_t>(page) * a.page_size + pos % a.page_size;
      }
      a.slots[x] = slot <= 0x7fffffff ? static_cast<int>(slot) : -1;
    }
    tok_sum += ct;
    page_sum += cp;
    __syncthreads();  // the next chunk overwrites the sums
  }
  for (int64_t x = tok_sum + me; x < a.num_tokens; x += step) a.slots[x] = -1;
  if (me == 0) {
    a.cu[a.B] = static_cast<int>(min(tok_sum, static_cast<int64_t>(0x7fffffff)));
    *a.free_out = static_cast<int>(max(count - page_sum, static_cast<int64_t>(-0x7fffffff)));
  }
}

// ---------------------------------------------------------------- appending rows to the pages
//
// A copy of row_elems elements from row rows[i] (or i) of k_new and v_new to row slots[i] of the
// pool; slots or rows outside their range are skipped. A thread moves 16 bytes of a row.
constexpr int kAppendThreads = 256;

// The E4M3 code nearest to x / s (ties to even, magnitudes past 448 to 448, NaN to NaN), two at a
// time. r = RN(1 / s); q = x r corrected once by its remainder is RN(x / s) (Markstein's division,
// 1990). Its 24 bits may fall on a border between two codes, or on the wrong side of one, where the
// quotient does not; the exact remainder says on which side of q the quotient lies, so q is turned
// into the quotient cut off towards zero with its last bit set where it is inexact (rounding to
// odd), and the conversion of that rounds the quotient itself.
__device__ __forceinline__ float quotient_to_odd(float x, float s, float r) {
  const float q0 = x * r;
  const float q1 = fmaf(fmaf(-q0, s, x), r, q0);
  const float rem = fmaf(-q1, s, x);
  int bits = __float_as_int(q1);
  if (rem != 0.f) bits = (bits + ((__float_as_int(rem) ^ __float_as_int(x)) >> 31)) | 1;
  // beyond 1024 the conversion saturates (or keeps NaN), whatever the last bits; -0 stays -0
  return copysignf(fabsf(q0) <= 1024.f ? __int_as_float(bits) : q0, x);
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__global__ void __launch_bounds__(kAppendThreads) kv_append_bf16_kernel(const AppendArgs a) {
  const bool is_v = blockIdx.y == 1;
  const uint16_t* src = is_v ? a.v_new : a.k_new;
  uint16_t* dst = static_cast<uint16_t*>(is_v ? a.v_pages : a.k_pages);
  const int64_t stride = is_v ? a.v_stride : a.k_stride;
  const int per_row = a.row_elems / 8;
  const int64_t total = static_cast<int64_t>(a.num_slots) * per_row;
  for (int64_t x = static_cast<int64_t>(blockIdx.x) * kAppendThreads + threadIdx.x; x < total;
       x += static_cast<int64_t>(gridDim.x) * kAppendThreads) {
    const int i = static_cast<int>(x / per_row), c = static_cast<int>(x % per_row);
    const int slot = a.slots[i], row = a.rows ? a.rows[i] : i;
    if (slot < 0 || slot >= a.pool_rows || row < 0 || row >= a.num_rows) continue;
    *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(slot) * a.row_elems + 8 * c) =
        *reinterpret_cast<const uint4*>(src + row * stride + 8 * c);
  }
}

__global__ void __launch_bounds__(kAppendThreads) kv_append_fp8_kernel(const AppendArgs a) {
  const bool is_v = blockIdx.y == 1;
  const uint16_t* src = is_v ? a.v_new : a.k_new;
  uint8_t* dst = static_cast<uint8_t*>(is_v ? a.v_pages : a.k_pages);
  const float* scale = is_v ? a.v_scale : a.k_scale;
  const int64_t stride = is_v ? a.v_stride : a.k_stride;
  const int per_row = a.row_elems / 8;
  const int64_t total = static_cast<int64_t>(a.num_slots) * per_row;
  for (int64_t x = static_cast<int64_t>(blockIdx.x) * kAppendThreads + threadIdx.x; x < total;
       x += static_cast<int64_t>(gridDim.x) * kAppendThreads) {
    const int i = static_cast<int>(x / per_row), c = static_cast<int>(x % per_row);
    const int slot = a.slots[i], row = a.rows ? a.rows[i] : i;
    if (slot < 0 || slot >= a.pool_rows || row < 0 || row >= a.num_rows) continue;
    const uint4 u = *reinterpret_cast<const uint4*>(src + row * stride + 8 * c);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t code[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float s0 = scale[8 * c + 2 * e], s1 = scale[8 * c + 2 * e + 1];
      code[e] = e4m3x2(quotient_to_odd(__uint_as_float(w[e] << 16), s0, __frcp_rn(s0)),
                       quotient_to_odd(__uint_as_float(w[e] & 0xffff0000u), s1, __frcp_rn(s1)));
    }
    *reinterpret_cast<uint2*>(dst + static_cast<int64_t>(slot) * a.row_elems + 8 * c) =
        make_uint2(code[0] | (code[1] << 16), code[2] | (code[3] << 16));
  }
}

}  // namespace

cudaError_t launch_tree_mask(const TreeMaskArgs& a, cudaStream_t stream) {
  tree_mask_kernel<<<a.num_seqs, kMaskThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv_plan(const PlanArgs& a, cudaStream_t stream) {
  const int blocks = min(152, (a.num_tokens + kPlanThreads - 1) / kPlanThreads);
  kv_plan_kernel<<<max(blocks, 1), kPlanThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t stream) {
  const int64_t total = static_cast<int64_t>(a.num_slots) * (a.row_elems / 8);
  const int64_t blocks = (total + kAppendThreads - 1) / kAppendThreads;
  const dim3 grid(static_cast<unsigned>(blocks < 152 * 8 ? blocks : 152 * 8), 2);
  if (a.k_scale)
    kv_append_fp8_kernel<<<grid, kAppendThreads, 0, stream>>>(a);
  else
    kv_append_bf16_kernel<<<grid, kAppendThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace bw
