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
// What bounds it: one row of p (and of q) a request, V values, and for few requests the latency of what follows one
// another: lengths, links and tokens, their probabilities, the walk, the row, its sums, the border. A cluster of CTAs
// takes a request, each a part of the row; all of them walk the tree alike and send one another their sums. 64 trees
// over 131072 tokens: 13.1 us with other rows each time, from memory (2.6 TB/s), 11.0 with rows in L2, of which the row
// takes 6 (with cluster barriers around the sums, a second pass over a warp's run for the border and the walk in 64 bits:
// 25 us). A request whose drafts are refused one by one takes a sum each, 4.8 us over 151007 tokens (1.8 of them the walk
// and the exchange; the rest the latency of the values' arithmetic at two warps a scheduler), which 40 drawn trees' 25.5 us
// with rows in L2, 32.8 from memory, end with. Not faster: 512 threads a CTA, rows through a deeper ring in shared memory, a
// cluster spread over the SMs, rows read to and fro. (Times in this file are with rows in L2 where nothing else is said.)
#include <type_traits>

#include "kernels.h"
#include "packed.cuh"
#include "ptx.cuh"

namespace bw {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxNodes = kTreeMaxNodes;
// An SM: four CTAs of 64 registers, so that 64 requests are under way at once; with draft probabilities two of 110 (40
// trees over 151007 tokens: three of 80 registers take 1.08 times as long, four, with spills, 1.33).
constexpr int ctas(bool drawn) { return drawn ? 2 : 4; }
constexpr int kBatch = 4;  // pieces of a row that a lane has under way (40 drawn trees: with 6 1.09 times as long, 8 1.10)

// Values in [0, 1] (NaN and negative ones: 0, larger ones: 1).
__device__ __forceinline__ float unit(float x) { return __saturatef(x); }

// A non-negative value x as a multiple of 2^-44: `big` 2^-22ths, `small` the rest. Adding 3 (1.5 * 2^-21) rounds to a
// multiple of 2^-22 (2^-44), which then stands in the last bits: `big` and `small` are those bits, 3's (1.5 * 2^-21's)
// still in them, and count from kBigBits and kSmallBits.
constexpr float kBig = 3.f, kSmall = 0x1.8p-21f;
constexpr uint32_t kBigBits = 0x40400000u, kSmallBits = 0x35400000u;
struct Fixed {
  uint32_t big, small;
};
constexpr int64_t kOne = 1ll << 44;
__device__ __forceinline__ int64_t whole(int big, int small) { return (static_cast<int64_t>(big) << 22) + small; }
__device__ __forceinline__ int64_t whole(Fixed f) {
  return whole(static_cast<int>(f.big - kBigBits), static_cast<int>(f.small - kSmallBits));
}

// Four values of r = max(p - A q, 0), A = a_hi + a_lo (kDrawn), or r = p, each as a multiple of 2^-44
template <bool kDrawn>
__device__ __forceinline__ void four(const float (&p)[4], const float (&q)[4], float a_hi, float a_lo, Fixed (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const pair_t x = pair(unit(p[2 * i]), unit(p[2 * i + 1]));
    pair_t s = x, lo = 0;
    if constexpr (kDrawn) {  // (also where A = 0 and q does not count: with a branch 1.06 times as long)
      const pair_t y = pair(unit(q[2 * i]), unit(q[2 * i + 1])), hi2 = pair(a_hi, a_hi);
      const pair_t m = mul(pair(-a_hi, -a_hi), y);                         // A q = -m + m_lo
      const pair_t m_lo = fma(pair(a_lo, a_lo), y, fma(hi2, y, m));
      s = add(x, m);
      const pair_t back = sub(s, x);                                       // x + m = s + what follows, exactly
      lo = sub(add(sub(x, sub(s, back)), sub(m, back)), m_lo);
    }
    const pair_t a = add(s, pair(kBig, kBig)), rest = add(sub(s, add(a, pair(-kBig, -kBig))), lo), b = add(rest, pair(kSmall, kSmall));
    const bool some0 = !kDrawn || first(s) > -first(lo), some1 = !kDrawn || second(s) > -second(lo);
    f[2 * i] = some0 ? Fixed{__float_as_uint(first(a)), __float_as_uint(first(b))} : Fixed{kBigBits, kSmallBits};
    f[2 * i + 1] = some1 ? Fixed{__float_as_uint(second(a)), __float_as_uint(second(b))} : Fixed{kBigBits, kSmallBits};
  }
}
__device__ __forceinline__ int64_t fixed(float p) {  // the same of one p
  const float x[4] = {p, 0.f, 0.f, 0.f};
  Fixed f[4];
  four<false>(x, x, 0.f, 0.f, f);
  return whole(f[0]);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// v to *p of the cluster's CTA `rank`, where its arrival counts as 8 bytes on *bar
__device__ __forceinline__ void send(int64_t* p, uint64_t* bar, uint32_t rank, int64_t v) {
  asm volatile(
      "{\n\t.reg .b32 ra, rb;\n\tmapa.shared::cluster.u32 ra, %0, %2;\n\tmapa.shared::cluster.u32 rb, %1, %2;\n\t"
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b64 [ra], %3, [rb];\n\t}" ::"r"(smem_u32(p)),
      "r"(smem_u32(bar)), "r"(rank), "l"(v)
      : "memory");
}
// floor(w x) of a number w in [0, 1), -0 among them
__device__ __forceinline__ int64_t part_of(float w, int64_t x) {
  const uint32_t bits = __float_as_uint(w), e = bits >> 23 & 255;
  const uint64_t m = e ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;  // w = m 2^-down, down at least 24
  const int down = 150 - static_cast<int>(e ? e : 1);
  const uint64_t lo = m * static_cast<uint64_t>(x), hi = __umul64hi(m, static_cast<uint64_t>(x));
  return static_cast<int64_t>(down < 64 ? lo >> down | hi << (64 - down) : down < 128 ? hi >> (down - 64) : 0);
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

// Piece `piece`, or 0 where it is not in front of `end`. kWhole: only pieces that lie in the row from end to end, and
// of a q whose pieces begin where p's do: one load under a condition, so that a batch's arithmetic is one block of code
// (40 drawn trees: with branches 1.14 times as long; without q, where there is little of it, 64 trees 11.0 us with and 11.3
// without).
template <bool kDrawn, bool kWhole>
__device__ __forceinline__ void load_piece(const Row& row, bool with_q, int piece, int end, float (&p)[4], float (&q)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) p[e] = q[e] = 0.f;
  if constexpr (kWhole) {
    const int e = 4 * piece - row.skip;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
    const bool in = piece < end && e >= 0 && e + 4 <= row.V;
    if (in) x = *reinterpret_cast<const float4*>(row.p + e);
    if (kDrawn && in && with_q) y = *reinterpret_cast<const float4*>(row.q + e);
    p[0] = x.x, p[1] = x.y, p[2] = x.z, p[3] = x.w;
    if (kDrawn) q[0] = y.x, q[1] = y.y, q[2] = y.z, q[3] = y.w;
  } else if (piece < end) {
    row.load(row.p, piece, true, p);
    if (kDrawn && with_q) row.load(row.q, piece, row.q_alike, q);
  }
}

// Pieces of a warp's run: whole turns of 32, the runs of a cluster's warps one behind the other.
__device__ __forceinline__ int run_of(int pieces, int cluster) { return (pieces + 32 * kWarps * cluster - 1) / (32 * kWarps * cluster) * 32; }

enum State { kSum, kReady };  // r has to be summed; the walk is over and r's sums are there

constexpr int kMaxGroups = 128;  // that a warp's run may have
static_assert(kVerifyMaxVocab / 4 + 2 <= 32 * kWarps * kMaxCluster * kMaxGroups, "groups");

struct Shared {
  uint64_t arrived[2];           // the CTAs' sums, of two sums in turns
  int64_t part[2][kMaxCluster];
  int64_t warp_sum[kWarps];
  int64_t group[kWarps][kMaxGroups];  // of 32 pieces each, a warp's run
  int parent[kMaxNodes];  // -1: not to be tried
  int token[kMaxNodes];
  float u[kMaxNodes], p[kMaxNodes], q[kMaxNodes];  // p and q: of the node's token behind its parent
  int path[kMaxNodes];
  int refused[kMaxNodes];  // different tokens refused behind the path's last node
  int count, num_refused, state, abort;
  float a_hi, a_lo;
};

template <bool kDrawn>
__global__ void __launch_bounds__(kThreads, ctas(kDrawn)) tree_verify_kernel(const VerifyArgs a, int cluster) {
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
  // rows behind the last request hold no node (up to 2^31 - 1 of them: a step past the last would leave 32 bits)
  if (b + 1 >= a.num_seqs)
    for (int64_t i = static_cast<int64_t>(behind) + rank * kThreads + tid; i < a.total_q; i += cluster * kThreads) a.accepted[i] = -1;
  if (n == 0) {  // the whole cluster leaves
    for (int64_t i = static_cast<int64_t>(t0) + rank * kThreads + tid; i < behind; i += cluster * kThreads) a.accepted[i] = -1;
    if (b < a.num_seqs && rank == 0 && tid == 0) {
      a.counts[b] = 0;
      a.next[b] = -1;
    }
    return;
  }
  if (tid == 0) {
    mbar_init(&sm.arrived[0], 1);
    mbar_init(&sm.arrived[1], 1);
    sm.abort = 0;
    sm.path[0] = 0;
    fence_mbar_init();
  }
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // waited for before the first sum is sent
  for (int i = tid; i < n; i += kThreads) {
    const int up = i > 0 ? a.parents[t0 + i] : -1, t = a.tokens[t0 + i];
    const bool real = up >= 0 && up < i && t >= 0 && t < a.vocab;
    sm.parent[i] = real ? up : -1;
    sm.token[i] = t;
    sm.u[i] = a.u[t0 + i];
    sm.p[i] = real ? unit(a.p[static_cast<int64_t>(t0 + up) * a.p_stride + t]) : 0.f;
    if (kDrawn) sm.q[i] = real ? unit(a.q[static_cast<int64_t>(t0 + up) * a.q_stride + t]) : 0.f;
  }
  __syncthreads();

  // the walk's state (warp 0, its lanes alike)
  int next = 1, last = 0, count = 1, refused = 0;
  // A = a_hi + a_lo; S as a double without draft probabilities, as a sum of integers with them (64-bit floats on the way from
  // a sum to the next one take a third of a microsecond)
  float a_hi = 0.f, a_lo = 0.f, Sf = 1.f;
  double S = 1.0;
  int64_t S_int = kOne;
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
            a_hi = a_lo = 0.f;
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
        // u S q < r in 32 bits, and in 64 only where they may be wrong: 64 take the walk six times as long
        const float u = sm.u[c], p = sm.p[c], q = kDrawn ? sm.q[c] : 1.f;
        bool again = false;  // the same token was refused before
        if constexpr (!kDrawn) {
          const int t = sm.token[c];
          for (int x = lane; x < refused; x += 32) again |= sm.refused[x] == t;
          again = __any_sync(0xffffffffu, again);
        }
        const float bar = u * Sf * q, r = again ? 0.f : kDrawn ? p - a_hi * q : p;
        bool keep = bar < r;
        if (!(fabsf(bar - r) > 0x1p-20f * (fabsf(bar) + p + a_hi * q))) {
          const double A = static_cast<double>(a_hi) + a_lo, sum = kDrawn ? static_cast<double>(S_int) * 0x1p-44 : S;
          const double rd = again ? 0.0 : kDrawn ? fmax(p - A * q, 0.0) : p;
          keep = u * sum * q < rd;
        }
        if (keep) {
          last = c;
          if (lane == 0) sm.path[count] = c;
          ++count;
          refused = 0;
          a_hi = a_lo = 0.f;
          S = 1.0, Sf = 1.f, S_int = kOne;
          summed = false;
        } else if constexpr (kDrawn) {
          // A += S, whose first 24 bits are Sf
          const float s_lo = static_cast<float>(S_int - static_cast<int64_t>(Sf * 0x1p44f)) * 0x1p-44f;
          const float t = a_hi + Sf, b = t - a_hi;  // a_hi + Sf = t + what follows, exactly
          const float lo = (a_hi - (t - b)) + (Sf - b) + (a_lo + s_lo);
          a_hi = t + lo;
          a_lo = lo - (a_hi - t);
          break;
        } else if (!again) {
          S = fmax(S - p, 0.0);
          Sf = static_cast<float>(S);
          if (lane == 0) sm.refused[refused] = sm.token[c];
          ++refused;
          __syncwarp();
        }
      }
      if (lane == 0) {
        sm.count = count;
        sm.num_refused = refused;
        sm.a_hi = a_hi;
        sm.a_lo = a_lo;
        sm.state = state;
      }
    }
    __syncthreads();
    if (sm.state == kReady) break;

    // ---- the sum of r: each warp of the cluster takes a run of pieces
    const Row row(a, t0 + sm.path[sm.count - 1]);
    const float A_hi = sm.a_hi, A_lo = sm.a_lo;
    const int run = run_of(row.pieces, cluster), v0 = min((rank * kWarps + warp) * run, row.pieces), v1 = min(v0 + run, row.pieces);
    mine = 0;
    const bool with_q = A_hi != 0.f;  // A = 0: r is p
    auto sum_run = [&](auto whole_pieces) {
      constexpr bool kWhole = decltype(whole_pieces)::value;
      float p[kBatch][4], q[kBatch][4];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) load_piece<kDrawn, kWhole>(row, with_q, v0 + 32 * i + lane, v1, p[i], q[i]);
      for (int v = v0; v < v1; v += 32 * kBatch) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          Fixed f[4];
          four<kDrawn>(p[i], q[i], A_hi, A_lo, f);
          load_piece<kDrawn, kWhole>(row, with_q, v + 32 * (i + kBatch) + lane, v1, p[i], q[i]);
          // (128 values are below 2^30 in either part)
          const int big = __reduce_add_sync(0xffffffffu, static_cast<int>(f[0].big + f[1].big + f[2].big + f[3].big - 4 * kBigBits));
          const int small =
              __reduce_add_sync(0xffffffffu, static_cast<int>(f[0].small + f[1].small + f[2].small + f[3].small - 4 * kSmallBits));
          const int64_t x = whole(big, small);
          const int g = (v - v0) / 32 + i;
          if (lane == 0 && 32 * g < v1 - v0) sm.group[warp][g] = x;
          mine += x;
        }
      }
    };
    if (kDrawn && (!with_q || row.q_alike)) {
      sum_run(std::true_type{});
      // the pieces that reach past the row, its first and its last
#pragma unroll 1
      for (int piece = row.skip ? 0 : row.pieces - 1; piece < row.pieces; piece += max(row.pieces - 1, 1)) {
        if (piece < v0 || piece >= v1 || (4 * piece >= row.skip && 4 * piece + 4 <= row.V + row.skip)) continue;
        float p[4], q[4];
        load_piece<kDrawn, false>(row, with_q, piece, v1, p, q);
        Fixed f[4];
        four<kDrawn>(p, q, A_hi, A_lo, f);
        const int64_t x = whole(f[0]) + whole(f[1]) + whole(f[2]) + whole(f[3]);
        if (lane == 0) sm.group[warp][(piece - v0) / 32] += x;
        mine += x;
      }
    } else {
      sum_run(std::false_type{});
    }
    if constexpr (!kDrawn) {
      __syncwarp();
      for (int x = 0; x < sm.num_refused; ++x) {
        const int t = sm.refused[x], piece = (t + row.skip) / 4;
        if (piece >= v0 && piece < v1) {
          const int64_t f = fixed(row.p[t]);
          mine -= f;
          if (lane == 0) sm.group[warp][(piece - v0) / 32] -= f;
        }
      }
    }
    if (lane == 0) sm.warp_sum[warp] = mine;
    __syncthreads();
    int64_t cta = 0;
    warps_before = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) warps_before = cta;
      cta += sm.warp_sum[w];
    }
    // Two sums' places and barriers in turns: a CTA sends a sum only when it has all of the one before, for
    // which every CTA has armed its barrier, and with that has seen the sum before that one.
    uint64_t* arrived = &sm.arrived[turn & 1];
    if (turn == 0) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // every CTA's barriers are there
    if (warp == 0) {
      mbar_arrive_expect_tx(arrived, 8 * cluster);
      __syncwarp();
      if (lane < cluster) send(&sm.part[turn & 1][rank], arrived, lane, cta);
    }
    const bool ok = mbar_wait(arrived, turn >> 1 & 1, a.timeout_ns, &sm.abort);
    if (!__syncthreads_and(ok)) {
      // The others may still send to this CTA, sums of this turn or of the next one: it stays until each of them has
      // ended or given up as well. That does not order what they sent before, so it stays for a millisecond more,
      // whatever its barriers say; a sum is under way for a microsecond or two.
      if (tid == 0) raise_timeout(&sm.abort, a.status);
      asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
      const uint64_t since = globaltimer_ns();
      for (int i = 0; i < 1 << 20 && globaltimer_ns() - since < 1000000; ++i) __nanosleep(500);
      return;
    }
    before = total = 0;
    for (int r = 0; r < cluster; ++r) {
      if (r == rank) before = total;
      total += sm.part[turn & 1][r];
    }
    summed = true;
    if (warp == 0) {
      if constexpr (kDrawn) {
        S_int = total;
        Sf = static_cast<float>(total) * 0x1p-44f;
      } else {
        S = static_cast<double>(total) * 0x1p-44;
        Sf = static_cast<float>(S);
      }
    }
  }

  if (rank == 0) {
    const int kept = sm.count;
    for (int64_t i = tid; i < behind - t0; i += kThreads) a.accepted[t0 + i] = i < kept ? t0 + sm.path[i] : -1;
    if (tid == 0) {
      a.counts[b] = kept;
      if (total == 0) a.next[b] = -1;  // p has no probabilities at all
    }
  }
  // ---- the first value whose running sum exceeds w times the sum: in one warp's run, one of its groups
  const float w = a.w[b];
  const int64_t bar = part_of(w >= 0.f ? fminf(w, 1.f - 0x1p-24f) : 0.f, total);
  int64_t sum = before + warps_before;
  if (!(sum <= bar && bar < sum + mine)) return;
  const Row row(a, t0 + sm.path[sm.count - 1]);
  const float A_hi = sm.a_hi, A_lo = sm.a_lo;
  const int run = run_of(row.pieces, cluster), v0 = min((rank * kWarps + warp) * run, row.pieces), v1 = min(v0 + run, row.pieces);
  auto scan = [&](int64_t x) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    return x;
  };
  int g = 0;
  for (;; g += 32) {  // (one of the run's groups holds it)
    const int64_t x = scan(32 * (g + lane) < v1 - v0 ? sm.group[warp][g + lane] : 0);
    const unsigned over = __ballot_sync(0xffffffffu, sum + x > bar);
    if (over || 32 * (g + 32) >= v1 - v0) {
      const int hit = over ? __ffs(over) - 1 : 31;
      sum += __shfl_sync(0xffffffffu, x, max(hit - 1, 0)) * (hit > 0);
      g += hit;
      break;
    }
    sum += __shfl_sync(0xffffffffu, x, 31);
  }
  float p[4], q[4];
  load_piece<kDrawn, false>(row, A_hi != 0.f, v0 + 32 * g + lane, v1, p, q);
  const int t = 4 * (v0 + 32 * g + lane) - row.skip;
  Fixed fixed4[4];
  four<kDrawn>(p, q, A_hi, A_lo, fixed4);
  int64_t f[4], all = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[e] = whole(fixed4[e]);
    if constexpr (!kDrawn)
      for (int k = 0; k < sm.num_refused; ++k)
        if (sm.refused[k] == t + e) f[e] = 0;
    all += f[e];
  }
  const int64_t upto = scan(all);
  const unsigned over = __ballot_sync(0xffffffffu, sum + upto > bar);
  if (over && lane == __ffs(over) - 1) {
    int64_t x = sum + upto - all;
    int e = 0;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      x += f[k];
      e += x <= bar;
    }
    a.next[b] = t + e;
  }
}

}  // namespace

cudaError_t launch_tree_verify(VerifyArgs& a, cudaStream_t stream) {
  cudaError_t e = status_word(&a.status);
  if (e != cudaSuccess) return e;
  a.timeout_ns = wait_timeout_ns();
  int dev = 0, sms = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  // CTAs a request: as many as keep a warp busy with some pieces of its row, fewer where there are many requests (what
  // a CTA does beside its part of the row is the same for all: 300 trees over 65536 tokens, 8 CTAs each 27.5 us, 4 19.6, 2
  // 16.1, 1 18.1; 100 drawn ones over 131072 36.6, 39.6, 54.1; 800 CTAs on 152 SMs), and enough to have places for the
  // sums of a row's groups
  constexpr int kPlaces = 32 * kWarps * kMaxGroups;
  const int most_ctas = 800 * sms / 152, pieces = a.vocab / 4 + 2;  // at most
  int cluster = kMaxCluster;
  while (cluster > 1 && (a.vocab < cluster * kWarps * 128 || a.num_seqs * cluster > most_ctas)) cluster /= 2;
  while (pieces > cluster * kPlaces) cluster *= 2;
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
