// Verification of drafted trees: which drafts a request keeps, and the token behind them, distributed as if
// every token had been drawn from the target's probabilities.
//
// From the root on, with p the target's distribution behind the path's last node and r = p, S = 1 at first,
// the node's children are tried in their order. A child with token t and random number u is
//   drawn from a distribution q:       kept iff u S q(t) < r(t), else r <- max(r - S q, 0), S <- sum r;
//   any (the most probable ones, say): kept iff u S < r(t), else S <- S - r(t), r(t) <- 0.
// With A the sum of the S so far, r = max(p - A q, 0) whatever the number of refusals (subtracting and cutting
// off at 0 step by step is subtracting everything and cutting off once), so a refusal costs one number, not a
// row. When no child is left to try, the token behind the path is the first whose running sum of r exceeds
// w sum r.
//
// Sums decide, so they must not depend on their order or lose what lies next to a border: a value is rounded
// to a multiple of 2^-44 once (r itself in two floats, whose error is far below), and integers are summed. 64 bits
// in place of that would be 64 times slower than the loads on this card.
//
// What bounds it: one row of p (and of q) a request, V values, and the latency of the walk for few requests.
// A cluster of CTAs takes a request, each a part of the row; all of them walk the tree alike, from values
// gathered at once, and exchange their sums through distributed shared memory.
#include "kernels.h"
#include "ptx.cuh"

namespace bw {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxNodes = kTreeMaxNodes;
constexpr int kBatch = 8;  // vectors of a row that a lane has under way

// Values in [0, 1] (NaN and negative ones: 0, larger ones: 1).
__device__ __forceinline__ float unit(float x) { return __saturatef(x); }

// A non-negative value hi + lo, lo far below hi, as a multiple of 2^-44: `big` 2^-22ths, `small` the rest. Adding
// 3 (1.5 * 2^-21) rounds to a multiple of 2^-22 (2^-44), which then stands in the last bits.
struct Fixed {
  int big, small;
};
__device__ __forceinline__ Fixed fixed(float hi, float lo) {
  const float a = hi + 3.f, rest = (hi - (a - 3.f)) + lo, b = rest + 0x1.8p-21f;
  return {__float_as_int(a) - __float_as_int(3.f), __float_as_int(b) - __float_as_int(0x1.8p-21f)};
}
__device__ __forceinline__ int64_t whole(Fixed f) { return (static_cast<int64_t>(f.big) << 22) + f.small; }

// max(p - A q, 0) with A = a_hi + a_lo
__device__ __forceinline__ Fixed residual(float p, float q, float a_hi, float a_lo) {
  const float m = __fmul_rn(a_hi, q), m_lo = fmaf(a_lo, q, fmaf(a_hi, q, -m));  // A q = m + m_lo
  const float s = __fsub_rn(p, m), back = __fsub_rn(s, p);
  const float err = __fadd_rn(__fsub_rn(p, __fsub_rn(s, back)), __fsub_rn(-m, back));  // p - m = s + err
  const float lo = err - m_lo;
  return s + lo > 0.f ? fixed(s, lo) : Fixed{0, 0};
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void store_remote(void* p, uint32_t rank, int64_t v) {
  asm volatile("{\n\t.reg .b32 ra;\n\tmapa.shared::cluster.u32 ra, %0, %1;\n\tst.shared::cluster.b64 [ra], %2;\n\t}" ::"r"(smem_u32(p)),
               "r"(rank), "l"(v)
               : "memory");
}

// One row (or, with draft probabilities, two) of V values, in pieces of 4 that begin on 16 bytes. The first and
// last pieces may reach past the row: those values are not read and count as 0.
struct Row {
  const float* p;   // the row's first value
  const float* q;   // or null
  int skip;         // values of the first piece before the row
  int V, pieces;
  bool q_alike;     // q's pieces begin on 16 bytes where p's do
  __device__ __forceinline__ Row(const VerifyArgs& a, int64_t row) {
    p = a.p + row * a.p_stride;
    q = a.q ? a.q + row * a.q_stride : nullptr;
    skip = static_cast<int>(reinterpret_cast<uintptr_t>(p) >> 2) & 3;
    q_alike = (static_cast<int>(reinterpret_cast<uintptr_t>(q) >> 2) & 3) == skip;
    V = a.vocab;
    pieces = (skip + V + 3) / 4;
  }
  __device__ __forceinline__ void load(const float* x, int piece, bool alike, float (&v)[4]) const {
    const int e = 4 * piece - skip;
    if (alike && e >= 0 && e + 4 <= V) {
      const float4 f = *reinterpret_cast<const float4*>(x + e);
      v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = e + i >= 0 && e + i < V ? x[e + i] : 0.f;
    }
  }
};

// Pieces of a warp's run: whole turns of 32, the runs of a cluster's warps one behind the other.
__device__ __forceinline__ int run_of(int pieces, int cluster) { return (pieces + 32 * kWarps * cluster - 1) / (32 * kWarps * cluster) * 32; }

template <bool kDrawn>
__device__ __forceinline__ void load_batch(const Row& row, int piece, int end, float (&p)[kBatch][4], float (&q)[kDrawn ? kBatch : 1][4]) {
#pragma unroll
  for (int i = 0; i < kBatch; ++i, piece += 32) {
#pragma unroll
    for (int e = 0; e < 4; ++e) p[i][e] = 0.f;
    if constexpr (kDrawn)
#pragma unroll
      for (int e = 0; e < 4; ++e) q[i][e] = 0.f;
    if (piece < end) {
      row.load(row.p, piece, true, p[i]);
      if constexpr (kDrawn) row.load(row.q, piece, row.q_alike, q[i]);
    }
  }
}

enum State { kSum, kReady };  // r has to be summed; the walk is over and r's sums are there

struct Shared {
  int64_t part[2][kMaxCluster];  // the CTAs' sums, of two sums in turns
  int64_t warp_sum[kWarps];
  int parent[kMaxNodes];  // -1: not to be tried
  int token[kMaxNodes];
  float u[kMaxNodes], p[kMaxNodes], q[kMaxNodes];  // p and q: of the node's token behind its parent
  int path[kMaxNodes];
  int refused[kMaxNodes];  // different tokens refused behind the path's last node
  int count, num_refused, state;
  double A;
};

template <bool kDrawn>
__global__ void __launch_bounds__(kThreads) tree_verify_kernel(const VerifyArgs a, int cluster) {
  __shared__ Shared sm;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_rank()), b = blockIdx.x / cluster;
  int t0 = 0, behind = 0;  // the request's first row and the one behind its last
  if (b < a.num_seqs) {
    t0 = min(max(a.cu_q[b], 0), a.total_q);
    behind = min(max(a.cu_q[b + 1], t0), a.total_q);
  }
  const int n = min(behind - t0, a.max_nodes);
  // rows behind the last request hold no node
  if (b + 1 >= a.num_seqs)
    for (int i = behind + rank * kThreads + tid; i < a.total_q; i += cluster * kThreads) a.accepted[i] = -1;
  if (n == 0) {  // the whole cluster leaves
    for (int i = t0 + rank * kThreads + tid; i < behind; i += cluster * kThreads) a.accepted[i] = -1;
    if (b < a.num_seqs && rank == 0 && tid == 0) {
      a.counts[b] = 0;
      a.next[b] = -1;
    }
    return;
  }
  for (int i = tid; i < n; i += kThreads) {
    const int up = i > 0 ? a.parents[t0 + i] : -1, t = a.tokens[t0 + i];
    const bool real = up >= 0 && up < i && t >= 0 && t < a.vocab;
    sm.parent[i] = real ? up : -1;
    sm.token[i] = t;
    sm.u[i] = a.u[t0 + i];
    sm.p[i] = real ? unit(a.p[static_cast<int64_t>(t0 + up) * a.p_stride + t]) : 0.f;
    if (kDrawn) sm.q[i] = real ? unit(a.q[static_cast<int64_t>(t0 + up) * a.q_stride + t]) : 0.f;
  }
  if (tid == 0) sm.path[0] = 0;
  __syncthreads();

  // the walk's state (warp 0, its lanes alike)
  int next = 1, last = 0, count = 1, refused = 0;
  double A = 0.0, S = 1.0;
  bool summed = false;  // the sums below are of r as it is now
  // r's sums: of the CTAs before this one, of all, of this CTA's warps before this one, of this warp
  int64_t before = 0, total = 0, warps_before = 0, mine = 0;
  bool whole_row = false;  // nothing was left of r: the token is drawn from p itself
  for (int turn = 0;; ++turn) {
    if (warp == 0) {
      State state = kSum;
      for (;;) {
        if (next >= n) {
          if (summed && (total != 0 || whole_row)) {
            state = kReady;
          } else if (summed) {
            whole_row = true;
            A = 0.0;
            refused = 0;
          }
          break;
        }
        const int first = next & ~31, j = first + lane;
        const unsigned hits = __ballot_sync(0xffffffffu, j >= next && j < n && sm.parent[min(j, kMaxNodes - 1)] == last);
        if (hits == 0) {
          next = first + 32;
          continue;
        }
        const int c = first + __ffs(hits) - 1;
        next = c + 1;
        double r = sm.p[c], bar = sm.u[c] * S;
        bool again = false;  // the same token was refused before
        if constexpr (kDrawn) {
          const double q = sm.q[c];
          r = fmax(r - A * q, 0.0);
          bar *= q;
        } else {
          const int t = sm.token[c];
          for (int x = lane; x < refused; x += 32) again |= sm.refused[x] == t;
          again = __any_sync(0xffffffffu, again);
          if (again) r = 0.0;
        }
        if (bar < r) {
          last = c;
          if (lane == 0) sm.path[count] = c;
          ++count;
          refused = 0;
          A = 0.0;
          S = 1.0;
          summed = false;
        } else if constexpr (kDrawn) {
          A += S;
          break;
        } else if (!again) {
          S = fmax(S - r, 0.0);
          if (lane == 0) sm.refused[refused] = sm.token[c];
          ++refused;
          __syncwarp();
        }
      }
      if (lane == 0) {
        sm.count = count;
        sm.num_refused = refused;
        sm.A = A;
        sm.state = state;
      }
    }
    __syncthreads();
    if (sm.state == kReady) break;

    // ---- the sum of r: each warp of the cluster takes a run of pieces
    const Row row(a, t0 + sm.path[sm.count - 1]);
    const float a_hi = static_cast<float>(sm.A), a_lo = static_cast<float>(sm.A - a_hi);
    const int run = run_of(row.pieces, cluster), v0 = min((rank * kWarps + warp) * run, row.pieces), v1 = min(v0 + run, row.pieces);
    mine = 0;
    for (int v = v0; v < v1; v += 32 * kBatch) {
      float p[kBatch][4], q[kDrawn ? kBatch : 1][4];
      load_batch<kDrawn>(row, v + lane, v1, p, q);
      Fixed sum{0, 0};
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const Fixed f = kDrawn ? residual(unit(p[i][e]), unit(q[i][e]), a_hi, a_lo) : fixed(unit(p[i][e]), 0.f);
          sum.big += f.big;
          sum.small += f.small;
        }
      mine += whole(sum);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, off);
    if constexpr (!kDrawn) {
      for (int x = 0; x < sm.num_refused; ++x) {
        const int t = sm.refused[x], piece = (t + row.skip) / 4;
        if (piece >= v0 && piece < v1) mine -= whole(fixed(unit(row.p[t]), 0.f));
      }
    }
    if (lane == 0) sm.warp_sum[warp] = mine;
    if (turn == 0)
      cluster_sync();  // every CTA runs, and may be written to
    else
      __syncthreads();
    int64_t cta = 0;
    warps_before = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) warps_before = cta;
      cta += sm.warp_sum[w];
    }
    // two sums' places in turns: whoever writes one has seen, by the barrier between, that all have read it
    if (tid < cluster) store_remote(&sm.part[turn & 1][rank], tid, cta);
    cluster_sync();
    before = total = 0;
    for (int r = 0; r < cluster; ++r) {
      if (r == rank) before = total;
      total += sm.part[turn & 1][r];
    }
    summed = true;
    S = static_cast<double>(total) * 0x1p-44;
  }

  if (rank == 0) {
    const int kept = sm.count;
    for (int i = tid; i < behind - t0; i += kThreads) a.accepted[t0 + i] = i < kept ? t0 + sm.path[i] : -1;
    if (tid == 0) {
      a.counts[b] = kept;
      if (total == 0) a.next[b] = -1;  // p has no probabilities at all
    }
  }
  // ---- the first value whose running sum exceeds w times the sum: in one warp's run, and there once more
  const float w = a.w[b];
  const double bar = static_cast<double>(w >= 0.f ? fminf(w, 1.f - 0x1p-24f) : 0.f) * static_cast<double>(total);
  int64_t sum = before + warps_before;
  if (!(static_cast<double>(sum) <= bar && bar < static_cast<double>(sum + mine))) return;
  const Row row(a, t0 + sm.path[sm.count - 1]);
  const float a_hi = static_cast<float>(sm.A), a_lo = static_cast<float>(sm.A - a_hi);
  const int run = run_of(row.pieces, cluster), v0 = min((rank * kWarps + warp) * run, row.pieces), v1 = min(v0 + run, row.pieces);
  for (int v = v0; v < v1; v += 32 * kBatch) {
    float p[kBatch][4], q[kDrawn ? kBatch : 1][4];
    load_batch<kDrawn>(row, v + lane, v1, p, q);
#pragma unroll 1
    for (int i = 0; i < kBatch; ++i) {
      // (the batch's values are picked by a loop so that its code stands here once)
      int64_t f[4], all = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x = 0.f, y = 0.f;
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (k == i) {
            x = p[k][e];
            if constexpr (kDrawn) y = q[k][e];
          }
        f[e] = whole(kDrawn ? residual(unit(x), unit(y), a_hi, a_lo) : fixed(unit(x), 0.f));
        if constexpr (!kDrawn) {
          const int t = 4 * (v + 32 * i + lane) - row.skip + e;
          for (int k = 0; k < sm.num_refused; ++k)
            if (sm.refused[k] == t) f[e] = 0;
        }
        all += f[e];
      }
      int64_t upto = all;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += x;
      }
      const unsigned over = __ballot_sync(0xffffffffu, static_cast<double>(sum + upto) > bar);
      if (over) {
        if (lane == __ffs(over) - 1) {
          int64_t x = sum + upto - all;
          int e = 0;
          for (; e < 3; ++e) {
            x += f[e];
            if (static_cast<double>(x) > bar) break;
          }
          a.next[b] = 4 * (v + 32 * i + lane) - row.skip + e;
        }
        return;
      }
      sum += __shfl_sync(0xffffffffu, upto, 31);
    }
  }
}

}  // namespace

cudaError_t launch_tree_verify(const VerifyArgs& a, cudaStream_t stream) {
  // CTAs a request: as many as keep a warp busy with some pieces of its row
  int cluster = kMaxCluster;
  while (cluster > 1 && a.vocab < cluster * kWarps * 128) cluster /= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.num_seqs > 0 ? a.num_seqs : 1) * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, a.q ? tree_verify_kernel<true> : tree_verify_kernel<false>, a, cluster);
}

}  // namespace bw
