// Paged KV cache bookkeeping on the GPU: ancestor masks of drafted token trees, block tables and
// slot maps from request lengths, and K/V rows written into the pages (bf16 or E4M3 codes).
#include <atomic>

#include "kernels.h"
#include "ptx.cuh"

namespace bw {

namespace {

constexpr int kSms = 152;  // of a GB300; it only says over how many blocks work is spread

// The first statement of every kernel here, a dependent launch: what the stream did before is complete and
// visible behind it. (Launched the ordinary way, a kernel behind another starts some 2.5 us later: 32768
// rows of 8 x 128 appended again and again 44.4 us a call, so 41.8.) The next kernel is set up when this
// one's blocks end, not when they start: a tree attention's CTAs that came in between them were spread over
// the SMs in another order, two with the same work on one, and took 84 to 89 us for 48 ragged requests.
__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---------------------------------------------------------------- tree masks
//
// mask[i] = mask[parent(i)] | bit i, position[i] = nk + depth(i), depth(i) = bits of mask[i] - 1. A
// parent precedes its children (anything else counts as a root), so the links have no cycle, and they
// are followed by doubling: with mask the nodes within 2^r - 1 steps up and up the node 2^r steps up,
// mask[i] |= mask[up[i]], up[i] = up[up[i]], until no node has one left: log2(depth) rounds whatever the
// tree (a walk per node took 5 us at depth 60, and as long as its longest line). One CTA per sequence, a
// thread per node, masks and links in shared memory; the new values are read before a barrier and
// written behind it.
constexpr int kMaskMaxNodes = kTreeMaxNodes;
constexpr int mask_smem(int threads, int words) { return threads * (8 * words + 2); }

template <int kWords>  // at least the call's words
__global__ void __launch_bounds__(kMaskMaxNodes) tree_mask_kernel(const TreeMaskArgs a) {
  wait_for_stream();
  extern __shared__ uint64_t sm_mask[];  // [kWords][threads], then int16_t up[threads]
  const int threads = blockDim.x, i = threadIdx.x;
  int16_t* up = reinterpret_cast<int16_t*>(sm_mask + static_cast<size_t>(kWords) * threads);
  const int seq = blockIdx.x;
  const int t0 = min(max(a.cu_q[seq], 0), a.total_q);
  const int n = min(min(max(a.cu_q[seq + 1], t0), a.total_q) - t0, a.max_nodes);
  const int base = a.nk ? a.nk[seq] : 0;
  int link = -1;
  if (i < n) {
    const int p = a.parents[t0 + i];
    if (p >= 0 && p < i) link = p;
  }
  uint64_t bits[kWords];
#pragma unroll
  for (int w = 0; w < kWords; ++w) {
    bits[w] = (i >> 6) == w ? 1ull << (i & 63) : 0;
    sm_mask[w * threads + i] = bits[w];
  }
  up[i] = static_cast<int16_t>(link);
  while (__syncthreads_or(link >= 0)) {
    int next = -1;
    if (link >= 0) {
#pragma unroll
      for (int w = 0; w < kWords; ++w) bits[w] |= sm_mask[w * threads + link];
      next = up[link];
    }
    __syncthreads();
    if (link >= 0) {
#pragma unroll
      for (int w = 0; w < kWords; ++w) sm_mask[w * threads + i] = bits[w];
      up[i] = static_cast<int16_t>(next);
    }
    link = next;
  }
  // the rows of the sequence are contiguous in a.mask: written in order from shared memory
  uint64_t* out = a.mask + static_cast<int64_t>(t0) * a.words;
  for (int x = i; x < n * a.words; x += threads) out[x] = sm_mask[x % a.words * threads + x / a.words];
  if (i < n && a.positions) {
    int depth = -1;
#pragma unroll
    for (int w = 0; w < kWords; ++w) depth += __popcll(bits[w]);
    a.positions[t0 + i] = base + depth;
  }
}

// ---------------------------------------------------------------- block tables and slot maps
//
// need_b = max(0, min(ceil((nk_b + new_b) / P), max_pages) - held_b) pages are taken from the top of
// the free stack, request after request: page k >= held_b of request b is
// free[count - 1 - (first_b + k - held_b)], first_b the sum of the needs before b. Every CTA scans
// all requests, kPlanThreads x kPlanRun at a time (two prefix sums; the tokens' in 64 bits, their sum may
// pass 32), and writes its share of the tokens' slots, of the new table entries and of the per-request
// outputs, so no CTA waits for another: a token's page is worked out from the old table or the free
// stack, never read from what this launch writes.
constexpr int kPlanThreads = 1024;
constexpr int kPlanRun = 2;
constexpr int kPlanChunk = kPlanThreads * kPlanRun;

__device__ __forceinline__ int plan_page(const PlanArgs& a, int count, int64_t i) {
  return i < count ? a.free_pages[count - 1 - i] : -1;  // past the stack: no page
}

__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(const PlanArgs a) {
  wait_for_stream();
  constexpr int kW = kPlanThreads / 32;
  // exclusive sums of the chunk's requests from its start, tokens cut off at the slots (`most`)
  __shared__ int s_tok[kPlanChunk], s_page[kPlanChunk], s_nk[kPlanChunk], s_held[kPlanChunk];
  __shared__ int64_t s_wt[kW];
  __shared__ int s_wp[kW];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int count = min(max(*a.free_count, 0), a.free_cap);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kPlanThreads;
  const int64_t me = static_cast<int64_t>(blockIdx.x) * kPlanThreads + tid;
  int64_t tok_sum = 0;
  int page_sum = 0;  // B x max_pages fits
  for (int b0 = 0, chunk = 0; b0 < a.B; b0 += kPlanChunk, ++chunk) {
    if (b0 > 0) __syncthreads();  // the last chunk's sums have been read
    int nk[kPlanRun], held[kPlanRun], need[kPlanRun], add[kPlanRun];
#pragma unroll
    for (int r = 0; r < kPlanRun; ++r) {
      const int b = b0 + tid * kPlanRun + r;
      nk[r] = b < a.B ? max(a.nk[b], 0) : 0;
      add[r] = b < a.B ? max(a.n_new[b], 0) : 0;
      held[r] = b < a.B ? min(max(a.held[b], 0), a.max_pages) : 0;
    }
    int64_t tok = 0;
    int page = 0;
#pragma unroll
    for (int r = 0; r < kPlanRun; ++r) {
      const int64_t keys = static_cast<int64_t>(nk[r]) + add[r];
      const int k32 = static_cast<int>(keys);  // rounded up without a sum that could pass 32 bits
      const int want = keys < static_cast<int64_t>(a.max_pages) * a.page_size ? k32 / a.page_size + (k32 % a.page_size != 0)
                                                                              : a.max_pages;
      need[r] = b0 + tid * kPlanRun + r < a.B ? max(want - held[r], 0) : 0;
      tok += add[r];
      page += need[r];
    }
    int64_t st = tok;  // inclusive sums over the warp, then the block
    int sp = page;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, st, off);
      const int y = __shfl_up_sync(0xffffffffu, sp, off);
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
    // the sums of the warps before this one, and of all, from a scan of the warps' totals by each warp
    int64_t vt = s_wt[lane];
    int vp = s_wp[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, vt, off);
      const int y = __shfl_up_sync(0xffffffffu, vp, off);
      if (lane >= off) {
        vt += x;
        vp += y;
      }
    }
    const int64_t chunk_tok = __shfl_sync(0xffffffffu, vt, 31);
    const int chunk_page = __shfl_sync(0xffffffffu, vp, 31);
    const int64_t before_t = __shfl_sync(0xffffffffu, vt, (warp + 31) & 31);
    const int before_p = __shfl_sync(0xffffffffu, vp, (warp + 31) & 31);
    if (warp > 0) {
      st += before_t;
      sp += before_p;
    }
    st -= tok;
    sp -= page;
    const int64_t most = min(chunk_tok, max(a.num_tokens - tok_sum, static_cast<int64_t>(0)));
#pragma unroll
    for (int r = 0; r < kPlanRun; ++r) {
      const int x = tid * kPlanRun + r, b = b0 + x;
      s_tok[x] = static_cast<int>(min(st, most));
      s_page[x] = sp;
      s_nk[x] = nk[r];
      s_held[x] = held[r];
      if (b < a.B && chunk % gridDim.x == blockIdx.x) {
        a.nk_out[b] = static_cast<int>(min(static_cast<int64_t>(nk[r]) + add[r], static_cast<int64_t>(0x7fffffff)));
        a.held_out[b] = held[r] + need[r];
        a.cu[b] = static_cast<int>(min(tok_sum + st, static_cast<int64_t>(0x7fffffff)));
      }
      st += add[r];
      sp += need[r];
    }
    __syncthreads();
    // the request of an item: the last one whose exclusive sum is at most the item's index
    auto request = [&](const int* sums, int x) {
      int lo = 0;
#pragma unroll
      for (int w = kPlanChunk / 2; w > 0; w >>= 1)
        if (sums[lo + w] <= x) lo += w;
      return lo;
    };
    for (int64_t x = me; x < chunk_page; x += step) {
      const int r = request(s_page, static_cast<int>(x));
      const int k = s_held[r] + (static_cast<int>(x) - s_page[r]);
      a.table[static_cast<int64_t>(b0 + r) * a.max_pages + k] = plan_page(a, count, static_cast<int64_t>(page_sum) + x);
    }
    for (int64_t x = me; x < most; x += step) {
      const int r = request(s_tok, static_cast<int>(x));
      const int64_t pos = static_cast<int64_t>(s_nk[r]) + (static_cast<int>(x) - s_tok[r]);
      int64_t slot = -1;
      if (pos < static_cast<int64_t>(a.max_pages) * a.page_size) {
        const int k = static_cast<int>(pos) / a.page_size;
        const int p = k < s_held[r] ? a.table[static_cast<int64_t>(b0 + r) * a.max_pages + k]
                                    : plan_page(a, count, static_cast<int64_t>(page_sum) + s_page[r] + (k - s_held[r]));
        if (p >= 0) slot = static_cast<int64_t>(p) * a.page_size + (static_cast<int>(pos) - k * a.page_size);
      }
      a.slots[tok_sum + x] = slot <= 0x7fffffff ? static_cast<int>(slot) : -1;
    }
    tok_sum += chunk_tok;
    page_sum += chunk_page;
  }
  for (int64_t x = tok_sum + me; x < a.num_tokens; x += step) a.slots[x] = -1;
  if (me == 0) {
    a.cu[a.B] = static_cast<int>(min(tok_sum, static_cast<int64_t>(0x7fffffff)));
    *a.free_out = count - page_sum;
  }
}

// ---------------------------------------------------------------- appending rows to the pages
//
// A copy of row_elems elements from row rows[i] (or i) of k_new and v_new to row slots[i] of the
// pool; slots or rows outside their range are skipped. A thread moves 16 bytes of a row.
//
// A thread keeps its channels (kVec of them, 16 bytes of output) and takes rows a grid apart, kRows to a
// batch. Slots are looked up two batches ahead and rows copied into shared memory one ahead, so the
// memory is busy while a batch is converted and stored. With E4M3 pages the reciprocals of the channels'
// scales stay in registers (reading and inverting the scales for every element took 47 us on 20001 rows of
// 8 x 128, dividing each element exactly 36 us, a bracket around each, with the rows in registers, 23.3, as
// here 21.9 us, 5.6 TB/s). The bytes bound the copy: 32768 rows of 8 x 128 in 40.9 us, 6.6 TB/s (rows in
// registers 42.5).
constexpr int kAppendThreads = 256;
constexpr int append_rows(bool fp8) { return fp8 ? 4 : 2; }
constexpr int append_smem(bool fp8) { return 2 * append_rows(fp8) * (fp8 ? 2 : 1) * kAppendThreads * 16; }

// The E4M3 code nearest to x / s (ties to even, magnitudes past 448 to 448, NaN to NaN). Rounding is
// monotonic, so where x r_lo and x r_hi, which bracket x / s, have the same code it is the quotient's:
// r_lo and r_hi are RN(1 / s) less and more 2^-22 of it, twice what the reciprocal and the product
// round together. Where the codes differ (one warp in some hundred) a border between two codes is near,
// and the quotient is rounded to odd: RN(x / s) may fall on a border, or on the wrong side of one, where
// the quotient does not; the exact remainder says on which side of it the quotient lies, so it is
// turned into the quotient cut off towards zero with its last bit set where it is inexact, and the
// conversion of that rounds the quotient itself. A power of two has an exact reciprocal and exact
// products, borders among them: r_lo = r_hi.
struct Bracket {
  float lo, hi;
};
__device__ __forceinline__ Bracket bracket(float s) {
  const float r = __frcp_rn(s);
  if ((__float_as_uint(s) & 0x7fffffu) == 0) return {r, r};
  if (r < 0x1p-126f) return {0.f, __int_as_float(0x7f800000)};  // too few bits left: always the quotient
  return {fmaf(r, -0x1p-22f, r), fmaf(r, 0x1p-22f, r)};
}
__device__ __noinline__ float quotient_to_odd(float x, float s) {
  if (s < 0x1p-64f) x *= 0x1p64f, s *= 0x1p64f;  // keeps the remainder above the smallest number
  const float q = __fdiv_rn(x, s);
  const float rem = fmaf(-q, s, x);
  int bits = __float_as_int(q);
  if (rem != 0.f) bits = (bits + ((__float_as_int(rem) ^ __float_as_int(x)) >> 31)) | 1;
  // beyond 1024 the conversion saturates (or keeps NaN), whatever the last bits; -0 stays -0
  return copysignf(fabsf(q) <= 1024.f ? __int_as_float(bits) : q, x);
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

template <bool kFp8>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendArgs a, int threads) {
  wait_for_stream();
  constexpr int kVec = kFp8 ? 16 : 8;
  constexpr int kLoads = kVec / 8;
  constexpr int kRows = append_rows(kFp8);
  const bool is_v = blockIdx.y == 1;
  const uint16_t* src = is_v ? a.v_new : a.k_new;
  uint8_t* dst = static_cast<uint8_t*>(is_v ? a.v_pages : a.k_pages);
  const int64_t stride = is_v ? a.v_stride : a.k_stride;
  const int per_row = a.row_elems / kVec;
  const int me = blockIdx.x * kAppendThreads + threadIdx.x, lane = threadIdx.x & 31;
  if (me - lane >= threads) return;  // a warp without rows
  const bool idle = me >= threads;   // `threads` is a multiple of per_row
  const int c = me % per_row, step = threads / per_row;
  const float* scale = (is_v ? a.v_scale : a.k_scale) + kVec * c;
  // two halves of a ring in shared memory: [2][kRows][warps][kLoads x 32] pieces of 16 bytes. A warp copies its
  // pieces in the order of their addresses (E4M3: a lane's two pieces are the copies of two other lanes; each
  // lane copying its own, every sector crossed from L2 twice: 32 us)
  extern __shared__ uint4 sm_rows[];
  auto place = [&](int half, int r) { return sm_rows + ((half * kRows + r) * kAppendThreads + (threadIdx.x - lane)) * kLoads; };
  struct Ids {
    int slot[kRows], row[kRows];
  };
  const int64_t stride_i = static_cast<int64_t>(step) * kRows;
  auto look_up = [&](Ids& d, int64_t i0) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int64_t i = i0 + static_cast<int64_t>(r) * step;
      const bool is = i < a.num_slots && !idle;
      d.slot[r] = is ? a.slots[i] : -1;
      d.row[r] = static_cast<int>(i);
      if (a.rows) d.row[r] = is ? a.rows[i] : -1;
    }
  };
  auto fetch = [&](Ids& d, int half) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (d.slot[r] >= a.pool_rows || d.row[r] < 0 || d.row[r] >= a.num_rows) d.slot[r] = -1;
#pragma unroll
      for (int q = 0; q < kLoads; ++q) {
        const int owner = kLoads == 1 ? lane : 16 * q + lane / 2, part = kLoads == 1 ? 0 : lane & 1;
        const int row = __shfl_sync(0xffffffffu, d.slot[r] >= 0 ? d.row[r] : -1, owner);
        const int col = (me - lane + owner) % per_row * kVec + 8 * part;
        if (row >= 0)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(place(half, r) + 32 * q + lane)),
                       "l"(src + row * stride + col)
                       : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  Bracket inv[kVec];
  auto store = [&](const Ids& d, int half) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (d.slot[r] < 0) continue;
      const int64_t at = static_cast<int64_t>(d.slot[r]) * a.row_elems + kVec * c;
      uint4 u[kLoads];
#pragma unroll
      for (int q = 0; q < kLoads; ++q) u[q] = place(half, r)[lane * kLoads + q];
      if constexpr (kFp8) {
        float x[kVec];
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          const uint4& w4 = u[e / 8];
          const uint32_t h = (e / 2) % 4 == 0 ? w4.x : (e / 2) % 4 == 1 ? w4.y : (e / 2) % 4 == 2 ? w4.z : w4.w;
          x[e] = __uint_as_float(e % 2 ? h & 0xffff0000u : h << 16);
        }
        uint32_t code[4], differ = 0;
#pragma unroll
        for (int e = 0; e < kVec; e += 4) {
          code[e / 4] = e4m3x2(x[e] * inv[e].lo, x[e + 1] * inv[e + 1].lo) |
                        (e4m3x2(x[e + 2] * inv[e + 2].lo, x[e + 3] * inv[e + 3].lo) << 16);
          differ |= code[e / 4] ^ (e4m3x2(x[e] * inv[e].hi, x[e + 1] * inv[e + 1].hi) |
                                   (e4m3x2(x[e + 2] * inv[e + 2].hi, x[e + 3] * inv[e + 3].hi) << 16));
        }
        if (differ) {
#pragma unroll
          for (int e = 0; e < kVec; e += 4)
            code[e / 4] = e4m3x2(quotient_to_odd(x[e], scale[e]), quotient_to_odd(x[e + 1], scale[e + 1])) |
                          (e4m3x2(quotient_to_odd(x[e + 2], scale[e + 2]), quotient_to_odd(x[e + 3], scale[e + 3])) << 16);
        }
        *reinterpret_cast<uint4*>(dst + at) = make_uint4(code[0], code[1], code[2], code[3]);
      } else {
        *reinterpret_cast<uint4*>(dst + 2 * at) = u[0];
      }
    }
  };
  int64_t i0 = me / per_row;
  Ids now, next;
  look_up(now, i0);
  look_up(next, i0 + stride_i);
  fetch(now, 0);
  if constexpr (kFp8) {
#pragma unroll
    for (int e = 0; e < kVec; e += 4) {
      const float4 v = *reinterpret_cast<const float4*>(scale + e);
      inv[e] = bracket(v.x), inv[e + 1] = bracket(v.y), inv[e + 2] = bracket(v.z), inv[e + 3] = bracket(v.w);
    }
  }
  // a batch's slots are looked up two batches ahead and its rows copied one ahead
#pragma unroll 1
  for (int half = 0;; half ^= 1) {
    Ids after;
    look_up(after, i0 + 2 * stride_i);
    fetch(next, half ^ 1);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncwarp();
    store(now, half);
    __syncwarp();  // the next turn's copies go over what other lanes have just read
    i0 += stride_i;
    if (__all_sync(0xffffffffu, i0 >= a.num_slots)) break;
    now = next;
    next = after;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// More than 48 KB of shared memory is asked for once per device (`set`: a bit each), and then the most that any
// call takes: the limit belongs to the kernel, and a call's own size would lower it between another call's
// setting and its launch.
template <typename K>
cudaError_t allow_smem(K kernel, int most, std::atomic<uint64_t>& set) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev >= 64 || !(set.load() >> dev & 1))) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e == cudaSuccess && dev < 64) set.fetch_or(1ull << dev);
  }
  return e;
}

}  // namespace

cudaError_t launch_tree_mask(const TreeMaskArgs& a, cudaStream_t stream) {
  const int threads = (a.max_nodes + 31) / 32 * 32;
  auto go = [&](auto kernel, int words) {
    return launch_dependent(kernel, dim3(a.num_seqs), threads, mask_smem(threads, words), stream, a);
  };
  if (a.words == 1) return go(tree_mask_kernel<1>, 1);
  if (a.words == 2) return go(tree_mask_kernel<2>, 2);
  static_assert(mask_smem(256, 4) <= 48 * 1024, "without allow_smem");
  if (a.words <= 4) return go(tree_mask_kernel<4>, 4);
  static std::atomic<uint64_t> set{0};
  const cudaError_t e = allow_smem(tree_mask_kernel<16>, mask_smem(kMaskMaxNodes, 16), set);
  return e == cudaSuccess ? go(tree_mask_kernel<16>, 16) : e;
}

cudaError_t launch_kv_plan(const PlanArgs& a, cudaStream_t stream) {
  const int blocks = min(kSms, a.num_tokens / kPlanThreads + 1);
  return launch_dependent(kv_plan_kernel, dim3(blocks), kPlanThreads, 0, stream, a);
}

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t stream) {
  const int per_row = a.row_elems / (a.k_scale ? 16 : 8);
  // E4M3: one block an SM for each of K and V, as a thread inverts 16 scales before its rows (20001 rows
  // of 8 x 128: 21.9 us, two blocks 24.4); a copy has nothing to set up and 32 even out the SMs (32768
  // rows: 40.9 us, 16 41.5). In whole rows, no more than there are rows.
  const int64_t most = static_cast<int64_t>(a.num_slots) * per_row;
  int64_t threads = kSms * (a.k_scale ? 1 : 32) * kAppendThreads / per_row * per_row;
  if (threads == 0) threads = per_row;
  if (threads > most) threads = most;
  const dim3 grid(static_cast<unsigned>((threads + kAppendThreads - 1) / kAppendThreads), 2);
  if (!a.k_scale)
    return launch_dependent(kv_append_kernel<false>, grid, kAppendThreads, append_smem(false), stream, a, static_cast<int>(threads));
  static std::atomic<uint64_t> set{0};
  const cudaError_t e = allow_smem(kv_append_kernel<true>, append_smem(true), set);
  if (e != cudaSuccess) return e;
  return launch_dependent(kv_append_kernel<true>, grid, kAppendThreads, append_smem(true), stream, a, static_cast<int>(threads));
}

}  // namespace bw
