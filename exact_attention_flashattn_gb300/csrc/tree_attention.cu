// Attention of a tree of drafted tokens over a KV cache: node i of sequence b sees every one of the
// sequence's nk context keys in the cache and the drafts j whose bit is set in its mask,
//   O = sum_j e^(s_j - m) v_j / l,  l = sum_j e^(s_j - m),  s_j = scale q.k_j,  LSE = m + ln l,
// in one pass over the keys with a running maximum m and sum l. A node that sees no key gets O = 0
// and LSE = -inf.
#include <math.h>

#include "kernels.h"
#include "ptx.cuh"

namespace bw {

namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ float bf16_f32(uint32_t bits) { return __uint_as_float(bits << 16); }

// One CTA per (node, query head): each warp takes every kWarps-th key, its lanes the channels.
template <int D>
__global__ void __launch_bounds__(kWarps * 32) tree_rows_kernel(const TreeArgs a) {
  constexpr int kC = D / 32;  // channels per lane: lane + 32 c
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.x, i = blockIdx.y, b = blockIdx.z;
  const int t0 = min(max(a.cu_q[b], 0), a.total_q);
  const int n = min(min(max(a.cu_q[b + 1] - t0, 0), a.total_q - t0), a.max_nodes);
  if (i >= n) return;
  const int nk = min(max(a.nk[b], 0), a.kv_cap), hkv = h / a.g;
  float q[kC], o[kC], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    q[c] = bf16_f32(a.q[(t0 + i) * a.q_stride + h * D + lane + 32 * c]) * a.scale_log2;
    o[c] = 0.f;
  }
  const uint64_t* bits = a.mask + static_cast<int64_t>(t0 + i) * a.mask_words;
  for (int j = warp; j < nk + n; j += kWarps) {
    const uint16_t *k, *v;
    if (j >= nk) {
      const int x = j - nk;
      if (!(bits[x >> 6] >> (x & 63) & 1)) continue;
      k = a.k_new + (t0 + x) * a.k_new_stride + hkv * D;
      v = a.v_new + (t0 + x) * a.v_new_stride + hkv * D;
    } else {
      int64_t row;
      if (a.block_table) {
        int page = a.block_table[static_cast<int64_t>(b) * a.max_pages + j / a.page_size];
        page = min(max(page, 0), a.num_pages - 1);
        row = (static_cast<int64_t>(page) * a.page_size + j % a.page_size) * a.Hkv + hkv;
      } else {
        row = (static_cast<int64_t>(b) * a.Hkv + hkv) * a.kv_cap + j;
      }
      k = a.k + row * D;
      v = a.v + row * D;
    }
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < kC; ++c) s = fmaf(q[c], bf16_f32(k[lane + 32 * c]), s);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    const float m_new = fmaxf(m, s), base = m_new == -INFINITY ? 0.f : m_new;
    const float f = ex2(m - base), p = ex2(s - base);
    m = m_new;
    l = l * f + p;
#pragma unroll
    for (int c = 0; c < kC; ++c) o[c] = o[c] * f + p * bf16_f32(v[lane + 32 * c]);
  }
  __shared__ float sm_m[kWarps], sm_l[kWarps], sm_o[kWarps][D];
  if (lane == 0) {
    sm_m[warp] = m;
    sm_l[warp] = l;
  }
#pragma unroll
  for (int c = 0; c < kC; ++c) sm_o[warp][lane + 32 * c] = o[c];
  __syncthreads();
  float M = -INFINITY, L = 0.f;
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w]);
  const float base = M == -INFINITY ? 0.f : M;
  for (int w = 0; w < kWarps; ++w) L += sm_l[w] * ex2(sm_m[w] - base);
  const int64_t orow = static_cast<int64_t>(t0 + i) * a.Hq + h;
  for (int c = threadIdx.x; c < D; c += kWarps * 32) {
    float x = 0.f;
    for (int w = 0; w < kWarps; ++w) x += sm_o[w][c] * ex2(sm_m[w] - base);
    a.o[orow * D + c] = static_cast<uint16_t>(pack_bf16x2(L == 0.f ? 0.f : x / L, 0.f));
  }
  if (a.lse && threadIdx.x == 0) a.lse[orow] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

}  // namespace

size_t tree_ws_bytes(int, int, int, int) { return 256; }

cudaError_t launch_tree(const TreeArgs& a, cudaStream_t stream) {
  const dim3 grid(a.Hq, a.max_nodes, a.num_seqs);
  if (a.d == 64) tree_rows_kernel<64><<<grid, kWarps * 32, 0, stream>>>(a);
  if (a.d == 128) tree_rows_kernel<128><<<grid, kWarps * 32, 0, stream>>>(a);
  if (a.d == 256) tree_rows_kernel<256><<<grid, kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace bw
