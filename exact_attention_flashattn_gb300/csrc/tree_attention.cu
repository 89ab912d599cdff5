// Attention of a tree of drafted tokens over a KV cache: node i of sequence b sees every one of the
// sequence's nk context keys in the cache and the drafts j whose bit is set in its mask,
//   O = sum_j e^(s_j - m) v_j / l,  l = sum_j e^(s_j - m),  s_j = scale q.k_j,  LSE = m + ln l,
// in one pass over the keys with a running maximum m and sum l (the recurrence of the prefill
// kernels). A node that sees no key gets O = 0 and LSE = -inf.
//
// What bounds it: the cache is read once, 4 d bytes per key and KV head, and every key costs 4 d
// operations per row, a row being one (node, query head) pair of the KV head's group. 128 rows are
// far on the memory side of this card (at d = 128, 128 keys x 128 rows take 0.67 us of one SM's tensor
// pipe, their K and V 1.5 us of its share of HBM), 256 rows about level with it. So a tile holds 128
// rows (whole nodes: kTreeRows / g of them, which the Q copy's box {64, g, nodes} lays out without a
// gather), and a unit of work is one row tile of one KV head, or two (kTiles == 2) when a sequence
// may have more than 128 rows, so that a cache byte serves up to 256.
//
// Split: lengths are on the device, and one long sequence has to fill the GPU as well as many short
// ones. The key tiles of all units form one list (unit after unit: tree_unit_cost places for what a unit
// costs beside its tiles, its context tiles, then its drafts), and CTA c of G takes places
// [c T / G, (c + 1) T / G), whatever the lengths (with pages, a group of CTAs, each for another KV head: the
// list is then of the units of head groups). A unit that lies within one CTA's range is finished there; otherwise each
// CTA that has a part of it writes its (m, l, o), at most two such parts per CTA, and a second,
// dependent launch merges them in the order of the keys, so results do not depend on which CTA ends first.
//
// Inside a CTA a stream has an S and an O in tensor memory, an MMA issuing warp and a softmax warpgroup
// (thread = row = TMEM lane):
//   kTiles == 2   two streams, one per row tile, reading the same K and V tiles; one CTA per SM.
//   kTiles == 1   one stream, two CTAs per SM: each has its own units, so one's hand-over from unit to
//                 unit runs beside the other's tiles (both in one CTA on one unit's even and odd tiles
//                 took 8 us a unit more). Where a tile has at most 64 rows, the second half of the CTAs
//                 puts them on lanes 64 to 127: a warp's softmax costs the same for one row as for 32, and
//                 so the two CTAs of an SM use all four of its sub-partitions.
//   d == 256      (O alone takes half of tensor memory) one stream of 64-key tiles, two S buffers, one
//                 CTA per SM.
// A stream's S -> softmax -> P.V is a serial chain per tile; two of them, out of step, cover it.
// Producer warps stream K and V tiles (TMA, 128-byte swizzle; from a paged cache one copy per run of
// rows inside a page, a lane each) through a ring of shared-memory slots that runs on across units.
// The tail tile of the context and the tiles of drafts may hold rows that do not count (keys past
// the end, other sequences' drafts) and values that some rows must not see; 0 * NaN would still
// reach O, so the issuing warp zeroes such V rows, and infinities and NaN in V rows of drafts, in
// shared memory before the P.V of the tile; rows that do see those get them back at the end.
// Every wait is bounded; a timed-out wait sets the device status word, the CTA stops producing
// output, waits for its own copies and MMAs and frees its TMEM.
//
// Chunks (kChunk): the new tokens' own K and V are in the cache too, and the mask is the causal one at the sequence's
// end, token i of nq seeing keys up to i + nk - nq. A chunk of thousands of tokens has many units, which end at their
// own last key; the tiles that all of a unit's rows see come first, through the loops without masks, then those on the
// diagonal. The operations bound it: 2 x 8192 tokens of 32/8 heads of 128 take 704 us, 1560 TFLOP/s, called on end
// 728 (as packed K and V 639), 512 tokens behind 65024 330 us, 1660 TFLOP/s, on end at the power cap 370. A batch mixes them with decode steps, of which a unit is one row
// tile: there both streams take it (even and odd key tiles, joined through tensor memory at its end), as one stream
// alone reads K and V at half the rate that HBM gives (40 requests, 60 % of them decode steps, 24/8 heads of 64: 238
// -> 222 us, now 213).
#include <math.h>

#include <atomic>
#include <type_traits>

#include "kernels.h"
#include "ptx.cuh"

namespace bw {

namespace {

constexpr float kRescaleThreshold = 8.0f;  // log2 units: o is rescaled when the max grew by more than 2^8
constexpr int kSegSlots = 4;
constexpr int kBarBytes = 1024;

template <int D, int kTiles>
struct Cfg {
  static constexpr int kStreams = kTiles;
  static constexpr int kKeys = D == 256 ? 64 : 128;  // keys per tile
  static constexpr int kHalves = D / 64;             // 128-byte swizzle atoms across the head dim
  static constexpr int kCtasPerSm = kTiles == 1 && D <= 128 ? 2 : 1;
  static constexpr uint32_t kQBytes = kTreeRows * D * 2;
  static constexpr uint32_t kTileBytes = kKeys * D * 2;
  // ring slots, which tiles of K and V take in turns: as many as fit
  static constexpr int kStages = kCtasPerSm == 2 ? (D == 64 ? 4 : 2) : (D == 64 ? 8 : 5);
  static constexpr uint32_t kRing = kTiles * kQBytes;
  static constexpr uint32_t kBar = kRing + kStages * kTileBytes;
  static constexpr uint32_t kMl = kBar + kBarBytes;  // chunks of two row tiles: stream 1's maxima and sums
  static constexpr uint32_t kSmem = kMl + (kTiles == 2 ? kTreeRows * 8 : 0) + 1024;  // + alignment slack
  static constexpr int kTmaWarp = 4 * kStreams;  // K tiles, Q and the list of segments
  static constexpr int kMmaWarp = kTmaWarp + 1;
  static constexpr int kTmaVWarp = kMmaWarp + kStreams;
  // a warp more that issues copies of K and V (with two row tiles the MMAs set the pace)
  static constexpr int kHelpers = kTiles == 1 ? 1 : 0;
  static constexpr int kWarps = kTmaVWarp + 1 + kHelpers;
  static constexpr int kThreads = 32 * kWarps;
  // S of a stream's next tile is issued ahead of the P.V of its current one where tensor memory has
  // the room: at d = 256 into the other S buffer, at d = 64 into the same one once the softmax has
  // read it, P having columns of its own
  static constexpr bool kTwoS = D == 256;
  static constexpr bool kSplitP = D == 64;
  static constexpr bool kLook = D != 128;
  // tensor memory columns; without kSplitP, P (bf16 pairs) takes the place of the S it was made from
  static constexpr uint32_t kCols = 512 / kCtasPerSm;
  static constexpr uint32_t kColS = D == 256 ? 256 : 0;                            // + kKeys a stream (or buffer)
  static constexpr uint32_t kColO = D == 256 ? 0 : 128 * kStreams;                 // + D a stream
  static constexpr uint32_t kColP = 128 * kStreams + D * kStreams;                 // kSplitP: + 64 a stream
  static constexpr uint32_t kColQ = 384;                                           // d = 256, chunks: Q, 128 columns
  static_assert(kSmem <= (kCtasPerSm == 2 ? 115712 : 232448), "shared memory");
  static_assert(kTiles == 1 || D <= 128, "tiles");
};

// A run of key tiles of one unit, published by the producer warp to the other roles.
struct Seg {
  int valid;        // 0: the CTA's list is exhausted
  int b;            // the sequence
  int tok0, nq, nk; // the sequence's first node, nodes, context keys
  int hkv, node0;   // KV head; first node (within the sequence) of the unit
  int k0, nt, ct;   // tiles [k0, k0 + nt) of the unit; its first ct tiles are context
  int slot;         // -1: the whole unit; else which of the CTA's two partial results
  int bad;          // set when a draft's V held an infinity or NaN
  int shift;        // chunks: node i sees keys up to and with i + shift (nk: the most that a row of the unit sees)
  int first;        // chunks: of the segment's tiles that all rows see whole, the one that is taken first (then the
                    // ones behind it, then those before)
  int split;        // chunks: the unit has one row tile, stream 0 takes its even key tiles, stream 1 the odd ones
};

struct Barriers {
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], p_full[2];
  uint64_t s_free[2];   // kSplitP: the softmax has read S
  uint64_t pv_done[2];  // kLook: the P.V of S buffer (stream) x has completed
  uint64_t turn[2];     // two row tiles at d = 128: P.V turns, 0: stream 0 to 1, 1: back
  uint64_t qt_full;     // chunks at d = 256: Q is in tensor memory
  uint64_t ml_full;     // split segments: stream 1's maxima, sums and O are there for stream 0
  uint64_t o_full[2], o_empty[2];
  uint64_t mma_done[2];
  uint64_t kv_full[8], kv_empty[8];
  uint64_t v_ready[8];  // two row tiles: stream 0 has looked over the V tile, in turn for those that need it
  uint64_t seg_full[kSegSlots], seg_empty[kSegSlots];
  Seg seg[kSegSlots];
  int scan[16], largest[16], smallest[16];
  int list[3];  // tiles of all sequences; the sequence of the CTA's first tile; tiles before it
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Barriers) <= kBarBytes, "barrier block");

__device__ __forceinline__ bool vote(bool x) { return __all_sync(0xffffffffu, x); }

// Places of the list that a tile takes. A batch of chunks mixes units of two row tiles with units of one (decode steps
// among them, whose tiles are a matter of their bytes): there a tile of two row tiles takes 4 places, of one 3, or at d =
// 64 with copies of more than 16 rows 2. 40 requests of up to 9000 keys, 60 % of them decode steps, 24/8 heads of 64, with
// 2 and with 3, in us: pages of 16 tokens 247 and 219, 48 (copies of 16 rows) 225 and 220, 80 (16) 223 and 219, 32 (32) 212
// and 219, 96 (32) 208 and 218, 64 208 and 219, 128 207 and 219; 24 requests of up to 20000 keys, 32/8 heads: 16 344 and
// 278, 48 311 and 279, 32 290 and 279, 96 277 and 278, 64 274 and 279, 128 266 and 279. 32/8 heads of 128, 16-token pages,
// up to 30000 keys: 723 with 3, 876 with 2 before both streams took such tiles.
template <int D, int kTiles, bool kChunk>
struct Places {
  static constexpr int kTile = kChunk && kTiles == 2 ? 4 : 1;
  static constexpr int kCost = tree_unit_cost(D) * kTile;
};

// Tiles of one sequence. Chunks: the units of its later rows have more of them, and the places of a KV head are
// summed unit by unit.
template <int D, int kTiles, bool kChunk>
struct SeqTiles {
  using P = Places<D, kTiles, kChunk>;
  int tok0, nq, nk;
  int ct, per_unit;  // context tiles, all tiles of a unit
  int row_units;     // units of a KV head
  int shift;         // chunks: as in Seg
  int places;        // chunks: of a KV head
  int largest, smallest;  // chunks: places of the largest and the smallest unit
  int single;        // chunks: places of a tile of one row tile
  // places of the list; the host bounds their sum
  __device__ __forceinline__ int all(int head_groups) const {
    return kChunk ? places * head_groups : (per_unit + P::kCost) * row_units * head_groups;
  }
  // chunks: keys that the last row of unit u sees, and the unit's tiles (one at least: rows without keys are written too)
  __device__ __forceinline__ int unit_keys(int u, int unit_nodes) const {
    return min(max(shift + min(nq, (u + 1) * unit_nodes), 0), nk);
  }
  template <int kKeys>
  __device__ __forceinline__ int unit_tiles(int u, int unit_nodes) const {
    const int n = unit_keys(u, unit_nodes);
    return max(n / kKeys + (n % kKeys != 0), 1);
  }
  // chunks: places of a tile of unit u, and of the unit
  __device__ __forceinline__ int weight(int u, int tile_nodes) const {
    return nq - u * kTiles * tile_nodes > tile_nodes ? P::kTile : single;
  }
  __device__ __forceinline__ int unit_places(int u, int tile_nodes) const {
    return unit_tiles<Cfg<D, kTiles>::kKeys>(u, kTiles * tile_nodes) * weight(u, tile_nodes) + P::kCost;
  }
  // chunks: sums over the units, by a lane, or by a converged warp whose lanes have the same sequence (a lane alone takes
  // 30 ns a unit: with its sums and its search for a CTA's first unit 3855 tokens of 5 heads of 128, 78 units, took 50.0
  // us, not 40.8; 16 prompts of 500 tokens, 32/8 heads of 128, 67.9 and 63.2)
  __device__ __forceinline__ void count(int tile_nodes, int from = 0, int step = 1) {
    places = largest = 0, smallest = 0x7fffffff;
#pragma unroll 1
    for (int u = from; u < row_units; u += step) {
      const int n = unit_places(u, tile_nodes);
      places += n, largest = max(largest, n), smallest = min(smallest, n);
    }
  }
  __device__ __forceinline__ void count_warp(int tile_nodes, int lane) {
    count(tile_nodes, lane, 32);
    places = __reduce_add_sync(0xffffffffu, places);
    largest = __reduce_max_sync(0xffffffffu, largest);
    smallest = __reduce_min_sync(0xffffffffu, smallest);
  }
};
template <int D, int kTiles, bool kChunk>
__device__ __forceinline__ SeqTiles<D, kTiles, kChunk> seq_tiles(const TreeArgs& a, int b) {
  constexpr int kKeys = Cfg<D, kTiles>::kKeys;
  SeqTiles<D, kTiles, kChunk> s;
  s.tok0 = min(max(a.cu_q[b], 0), a.total_q);
  s.nq = min(min(max(a.cu_q[b + 1], s.tok0), a.total_q) - s.tok0, a.max_nodes);
  s.nk = min(max(a.nk[b], 0), a.kv_cap);
  s.ct = s.nk / kKeys + (s.nk % kKeys != 0);
  s.per_unit = s.ct + (s.nq + kKeys - 1) / kKeys;
  const int unit_nodes = kTiles * a.tile_nodes;
  s.row_units = s.nq <= unit_nodes ? s.nq > 0 : (s.nq + unit_nodes - 1) / unit_nodes;  // 0 for a sequence without nodes
  if constexpr (kChunk) {
    s.shift = a.causal ? s.nk - s.nq : s.nk - 1;  // (its sum with nq fits: the host sees to that)
    s.single = Places<D, kTiles, kChunk>::kTile == 1 ? 1 : D == 64 && a.piece > 16 ? 2 : 3;
  }
  return s;
}

// T places over at most `most` CTAs, none with fewer than a tile's: the first T % G CTAs take one more.
struct Share {
  int G, per, rem;
  __device__ __forceinline__ Share(int T, int most, int tile) {
    G = max(min(T / tile, most), 1);
    per = T / G;
    rem = T - per * G;
  }
  __device__ __forceinline__ int begin(int c) const { return c * per + min(c, rem); }
  __device__ __forceinline__ int owner(int x) const {
    const int t = rem * (per + 1);
    return x < t ? x / (per + 1) : rem + (x - t) / per;
  }
};

// One copy by the calling lane (the wrapper in ptx.cuh elects one lane of a converged warp).
__device__ __forceinline__ void tma_load_3d_lane(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
      "[%2];\n" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// One MMA D[tmem] (+)= A[tmem] B[smem], issued by one lane of a converged warp.
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t blo, uint32_t bhi, uint32_t idesc,
                                        uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, pe;\n\t.reg .b64 db;\n\telect.sync _|pe, 0xffffffff;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tmov.b64 db, {%2, %3};\n\t"
      "@pe tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "r"(blo), "r"(bhi), "r"(idesc), "r"(acc)
      : "memory");
}

// The infinities and NaN in rows `from` to `valid` of a V tile in shared memory, [atom][kKeys rows][128 bytes], become
// zero. A converged warp.
template <int kHalves, int kKeys>
__device__ __forceinline__ void zero_bad(uint8_t* tile, int from, int valid, int lane) {
#pragma unroll 1
  for (int hf = 0; hf < kHalves; ++hf) {
#pragma unroll 1
    for (int off = from * 128 + lane * 16; off < valid * 128; off += 512) {
      uint4* at = reinterpret_cast<uint4*>(tile + hf * (kKeys * 128) + off);
      const uint4 v = *at;
      uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if ((w[e] & 0x7f80u) == 0x7f80u) w[e] &= 0xffff0000u;
        if ((w[e] & 0x7f800000u) == 0x7f800000u) w[e] &= 0xffffu;
      }
      *at = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}
// The same, and whether there were any. Values are looked over by products with 0, whose sum is 0 or NaN, eight pieces
// of 16 bytes a lane at a time: the last P.V of a unit waits for it (with compares, four pieces at a time, 128 rows at
// d = 128 took 3 us). Out of line, as in the issuing warp's loop it cost every tile 1 to 2 %.
template <int kHalves, int kKeys>
__device__ __noinline__ bool scan_v(uint8_t* tile, int from, int valid, int lane) {
  constexpr int kRun = 8 / kHalves;
  const int end = valid * 128;
  uint32_t sum[4] = {0u, 0u, 0u, 0u};
#pragma unroll 1
  for (int off = from * 128 + lane * 16; off < end; off += 512 * kRun) {
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = off + 512 * (i / kHalves);
      v[i] = at < end ? *reinterpret_cast<const uint4*>(tile + i % kHalves * (kKeys * 128) + at) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum[0]) : "r"(v[i].x), "r"(0u));
      asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum[1]) : "r"(v[i].y), "r"(0u));
      asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum[2]) : "r"(v[i].z), "r"(0u));
      asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum[3]) : "r"(v[i].w), "r"(0u));
    }
  }
  const bool bad = __any_sync(0xffffffffu, ((sum[0] | sum[1] | sum[2] | sum[3]) & 0x7fff7fffu) != 0);
  if (bad) zero_bad<kHalves, kKeys>(tile, from, valid, lane);
  return bad;
}
// V tile in shared memory: rows from `valid` to the next 16 become zero, and with `scan` the infinities and NaN of the
// others from row `from` on (returns whether there were any). A converged warp.
template <int kHalves, int kKeys>
__device__ __forceinline__ bool clean_v(uint8_t* tile, int from, int valid, bool scan, int lane) {
  const bool bad = scan && scan_v<kHalves, kKeys>(tile, from, valid, lane);
#pragma unroll
  for (int hf = 0; hf < kHalves; ++hf)
    for (int off = valid * 128 + lane * 16; off < (valid + 15) / 16 * 2048; off += 512)
      *reinterpret_cast<uint4*>(tile + hf * (kKeys * 128) + off) = make_uint4(0u, 0u, 0u, 0u);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the tensor pipe reads the tile
  __syncwarp();
  return bad;
}

// Registers: a softmax thread holds a row's 128 scores, the other four warps little; at d = 256 a row has 64
// and all have enough. A block's threads share what they were launched with: 256 x 128 (two on an SM) or
// 384 x 168.
template <int D, int kTiles>
struct Regs {
  static constexpr bool kSplit = D <= 128;
  static constexpr int kSoft = kTiles == 1 ? 184 : 192, kOther = kTiles == 1 ? 72 : 112;
  static_assert(!kSplit || kTiles * 128 * kSoft + 128 * kOther <= (kTiles == 1 ? 256 * 128 : 384 * 168), "register split");
  static __device__ __forceinline__ void give() {
    if constexpr (kSplit) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOther));
  }
  static __device__ __forceinline__ void take() {
    if constexpr (kSplit) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoft));
  }
};

// Softmax of a row's tile in which not every key counts: the context's last tile (the first `left` keys)
// and the tiles of drafts (those of them whose bit is set, from bit `bit0` of `bits` on; null: no mask). 32
// keys at a time and no further than the last that counts, S read twice, for the maximum and for the
// weights; P of chunk c goes to columns 16 c on, over S that has been read if that is where it goes.
// Out of line: few tiles take it, and in the loop its code and registers cost the others 10 to 30 %.
// Returns the new reference maximum, the sum of the weights and the factor for l and o.
struct MaskedTile {
  float m, l, alpha;
};
// Chunks: no mask, the row's own first `mine` keys. (Weights are rounded to bf16 as in the loop's own tiles, and for the same
// reason; l sums them before.)
template <bool kChunk>
__device__ __noinline__ MaskedTile masked_tile(uint32_t tS, uint32_t tP, int left, int mine, const uint64_t* bits, int bit0, float sl2,
                                               float m_ref) {
  const int chunks = (left + 31) / 32;
  auto load = [&](int c, uint32_t (&v)[32]) {
    const int rest = (kChunk ? mine : left) - 32 * c, bit = bit0 + 32 * c;
    uint32_t keep = rest >= 32 ? 0xffffffffu : kChunk && rest <= 0 ? 0u : (1u << rest) - 1u;
    if (!kChunk && bits) keep &= static_cast<uint32_t>(bits[bit >> 6] >> (bit & 32));
    tmem_ld32(tS + 32 * c, v);
    tmem_wait_ld();
    tmem_reg_fence(v);
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (!(keep >> e & 1)) v[e] = __float_as_uint(-INFINITY);
  };
  float mt = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < chunks; ++c) {
    uint32_t v[32];
    load(c, v);
#pragma unroll
    for (int e = 0; e < 32; e += 2) mt = max3f(mt, __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
  }
  MaskedTile r{m_ref, 0.f, 1.f};
  const float m_new = fmaxf(m_ref, mt * sl2);
  if (m_new > m_ref + kRescaleThreshold) {
    r.alpha = (m_ref == -INFINITY) ? 0.f : ex2(m_ref - m_new);
    r.m = m_new;
  }
  const float nm = (r.m == -INFINITY) ? 0.f : -r.m;
  float l0 = 0.f, l1 = 0.f;
#pragma unroll 1
  for (int c = 0; c < chunks; ++c) {
    uint32_t v[32], pk[16];
    load(c, v);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float x0, x1;
      ffma2(x0, x1, __uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]), sl2, nm);
      const float p0 = ex2(x0), p1 = ex2(x1);
      fadd2(l0, l1, p0, p1);
      pk[e] = pack_bf16x2(p0, p1);
    }
    tmem_st16(tP + 16 * c, pk);
  }
  r.l = l0 + l1;
  return r;
}

// Chunks: a warp's rows of O, in tensor memory from column tO on, times inv to rows `row` of `out` (-1: none). Rows are
// written four lanes to one, 64 bytes of it: each four lanes exchange their rows' pieces, and piece x of row k of the
// four goes to lane x's k-th store. (A lane's own row in pieces of 16 bytes, a store touches 32 rows, and a unit's end
// took 3 us.) Out of line, as its registers would make the loops over tiles spill.
template <int D>
__device__ __noinline__ void write_rows(uint32_t tO, float inv, int64_t row, uint16_t* out, int lane) {
#pragma unroll 1
  for (int c = 0; c < D / 32; ++c) {
    uint32_t o[32];
    tmem_ld32(tO + c * 32, o);
    tmem_wait_ld();
    tmem_reg_fence(o);
    auto two = [&](int e) { return pack_bf16x2(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv); };
    uint4 v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = make_uint4(two(8 * q), two(8 * q + 2), two(8 * q + 4), two(8 * q + 6));
    auto exchange = [&](uint4& low, uint4& high, int bit) {
      const bool upper = lane & bit;
      const uint4 give = upper ? low : high;
      const uint4 got = make_uint4(__shfl_xor_sync(0xffffffffu, give.x, bit), __shfl_xor_sync(0xffffffffu, give.y, bit),
                                   __shfl_xor_sync(0xffffffffu, give.z, bit), __shfl_xor_sync(0xffffffffu, give.w, bit));
      (upper ? low : high) = got;
    };
    exchange(v[0], v[1], 1);
    exchange(v[2], v[3], 1);
    exchange(v[0], v[2], 2);
    exchange(v[1], v[3], 2);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t to = __shfl_sync(0xffffffffu, row, (lane & ~3) + k);
      if (to >= 0) *reinterpret_cast<uint4*>(out + to * D + c * 32 + 8 * (lane & 3)) = v[k];
    }
  }
}

template <int D, int kTiles, bool kChunk>
__global__ void __launch_bounds__(Cfg<D, kTiles>::kThreads, Cfg<D, kTiles>::kCtasPerSm)
    tree_kernel(const __grid_constant__ TreeArgs a) {
  using C = Cfg<D, kTiles>;
  using P = Places<D, kTiles, kChunk>;
  // Chunks at d = 256, which are bound by their products: the softmax threads copy Q into tensor memory, where S reads
  // only K's 2 KB a step from shared memory, not Q's 4 KB too (2 x 8192 tokens, 16/4 heads: 977 us with Q read there).
  constexpr bool kQt = kChunk && D == 256;
  constexpr int kStreams = C::kStreams, kKeys = C::kKeys, kStages = C::kStages, kVSlots = (kStages + 1) / 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sRing = smem + C::kRing;
  Barriers* bar = reinterpret_cast<Barriers*>(smem + C::kBar);
  const int group = static_cast<int>(blockIdx.x) / a.head_group;  // of CTAs with the same places
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  if (warp == C::kTmaWarp && lane == 0) {
    prefetch_tmap(&a.tm_q);
    prefetch_tmap(&a.tm_k);
    prefetch_tmap(&a.tm_v);
    if constexpr (!kChunk) {
      prefetch_tmap(&a.tm_kn);
      prefetch_tmap(&a.tm_vn);
    }
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->q_full[i], 1);
      mbar_init(&bar->q_empty[i], 1);
      mbar_init(&bar->s_full[i], 1);
      mbar_init(&bar->p_full[i], kTreeRows);
      mbar_init(&bar->s_free[i], kTreeRows);
      mbar_init(&bar->pv_done[i], 1);
      mbar_init(&bar->turn[i], 1);
      mbar_init(&bar->o_full[i], 1);
      mbar_init(&bar->o_empty[i], kTreeRows);
      mbar_init(&bar->mma_done[i], 1);
    }
    mbar_init(&bar->qt_full, kTreeRows);
    mbar_init(&bar->ml_full, kTreeRows);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bar->kv_full[i], a.block_table ? 1 + C::kHelpers : 1);  // everyone who loads into the slot
      mbar_init(&bar->kv_empty[i], kTiles);  // one commit per stream that reads the slot
      mbar_init(&bar->v_ready[i], 1);
    }
    for (int i = 0; i < kSegSlots; ++i) {
      mbar_init(&bar->seg_full[i], 1);
      mbar_init(&bar->seg_empty[i], 5 * kStreams + 1 + C::kHelpers);  // all but the K producer
    }
    bar->abort = 0;
    fence_mbar_init();
  }
  // What the stream did before is complete and visible from here on. No tensor memory is held while
  // waiting: a CTA of the kernel before, beside this one, may have yet to take its own.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp == C::kMmaWarp) {
    tmem_alloc(&bar->tmem_base, C::kCols);
    tmem_relinquish();
  }

  // ---- the list of tiles: a thread sums the tiles of a run of sequences. Up to 128 sequences the
  // producer warp does it alone (nobody else needs the list), beyond that the whole block
  const bool wide = a.num_seqs > 128;
  const int run = wide ? (a.num_seqs + C::kThreads - 1) / C::kThreads : (a.num_seqs + 31) / 32;
  const int run0 = min((wide ? tid : lane) * run, a.num_seqs), run1 = min(run0 + run, a.num_seqs);
  int mine = 0, incl = 0, largest = 0, smallest = 0x7fffffff;
  if (wide || warp == C::kTmaWarp) {
    if constexpr (!kChunk) {
#pragma unroll 4
      for (int b = run0; b < run1; ++b) mine += seq_tiles<D, kTiles, kChunk>(a, b).all(a.head_groups);
    } else {
#pragma unroll 1
      for (int i = 0; i < run; ++i) {
        auto q = seq_tiles<D, kTiles, kChunk>(a, min(run0 + i, a.num_seqs - 1));
        if (run0 + i >= run1) q.row_units = 0;
        // sequences of many units by the whole warp, one after the other
        const unsigned many = __ballot_sync(0xffffffffu, q.row_units > 8);
        if (!(many >> lane & 1)) q.count(a.tile_nodes);
        for (unsigned left = many; left; left &= left - 1) {
          const int from = __ffs(left) - 1;
          auto x = q;
          x.nq = __shfl_sync(0xffffffffu, q.nq, from), x.nk = __shfl_sync(0xffffffffu, q.nk, from);
          x.shift = __shfl_sync(0xffffffffu, q.shift, from), x.row_units = __shfl_sync(0xffffffffu, q.row_units, from);
          x.count_warp(a.tile_nodes, lane);
          if (lane == from) q.places = x.places, q.largest = x.largest, q.smallest = x.smallest;
        }
        mine += q.all(a.head_groups);
        largest = max(largest, q.largest), smallest = min(smallest, q.smallest);
      }
      largest = __reduce_max_sync(0xffffffffu, largest);
      smallest = __reduce_min_sync(0xffffffffu, smallest);
    }
    incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += x;
    }
    if (wide && lane == 31) bar->scan[warp] = incl, bar->largest[warp] = largest, bar->smallest[warp] = smallest;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // the merge may be set up from now on; it waits for this grid to complete (not before this CTA has its
  // tensor memory, for the same reason)
  asm volatile("griddepcontrol.launch_dependents;");
  int my_begin = 0, my_end = 0;  // the group's places
  // Chunks: a unit that several CTAs share costs them their parts and the merge, about what 8 tiles take (16 at d = 256).
  // Where the largest unit is no longer than that and a share together (or, where several units may begin in a share,
  // than that alone), the CTA in whose share a unit begins takes it whole: 32 requests of 500 keys and one token,
  // d = 128, 25.4 -> 20.3 us, 4 of 1000 and 128 tokens 33.8 -> 30.5, 8 of 600 and 200 at d = 256 46.9 -> 41.0. With 12
  // tiles in place of 8, 4 of 1000 keys and 64 tokens took 28.7 us, not 24.3.
  bool whole_units = false;
  if (wide || warp == C::kTmaWarp) {
    int T = __shfl_sync(0xffffffffu, incl, 31), before = incl - mine;
    if (wide) {
      T = 0;
      for (int w = 0; w < C::kWarps; ++w) {
        if (w == warp) before += T;
        T += bar->scan[w];
        if (kChunk) largest = max(largest, bar->largest[w]), smallest = min(smallest, bar->smallest[w]);
      }
    }
    const Share share(T, a.groups, P::kTile);
    if (group < share.G && T > 0) my_begin = share.begin(group), my_end = share.begin(group + 1);
    if constexpr (kChunk) {
      constexpr int kMerge = (D == 256 ? 16 : 8) * P::kTile;  // what the parts and the merge take, in places
      whole_units = largest <= kMerge + (share.per <= smallest ? share.per : 0);
    }
    if (my_begin < my_end && before <= my_begin && my_begin < before + mine) {
      int b = run0;
      if constexpr (!kChunk)  // (chunks: the producer goes on from the thread's first sequence)
        for (int n; my_begin >= before + (n = seq_tiles<D, kTiles, kChunk>(a, b).all(a.head_groups)); ++b) before += n;
      bar->list[1] = b;
      bar->list[2] = before;
    }
    if (wide ? tid == 0 : lane == 0) bar->list[0] = T;
    if (wide)
      __syncthreads();
    else
      __syncwarp();
  }
  const uint32_t tbase = __shfl_sync(0xffffffffu, bar->tmem_base, 0);
  volatile int* abort = &bar->abort;
  const uint64_t tmo = a.timeout_ns;
  const int tile_nodes = a.tile_nodes;
  // TMEM lane of a tile's first row
  const int first_lane = a.tile_rows == 64 && 2 * blockIdx.x >= gridDim.x ? 64 : 0;
  const int no_abort = 0;

  // consumer side of the segment queue, called by a converged warp
  auto wait_seg = [&](int k) -> Seg* {
    return vote(mbar_wait(&bar->seg_full[k % kSegSlots], (k / kSegSlots) & 1, tmo, abort)) ? &bar->seg[k % kSegSlots] : nullptr;
  };
  auto release_seg = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar->seg_empty[k % kSegSlots]);
  };
  // chunks: keys that every row of the unit sees, and its first tile that some row does not see whole
  auto all_see = [&](const Seg& s) { return min(max(s.shift + s.node0 + 1, 0), s.nk); };
  auto first_masked = [&](const Seg& s) { return all_see(s) / kKeys; };
  // rows of the unit's row tile w that exist
  auto tile_rows = [&](const Seg& s, int w) { return max(0, min(tile_nodes, s.nq - s.node0 - w * tile_nodes)) * a.g; };

  // paged: the copy of a tile (atom copy % kHalves of piece copy / kHalves) that is this lane's; with a
  // helper, of each three the first two are the producer's
  auto share_copy = [&](int member) {
    if (C::kHelpers == 0) return lane;
    return member > 0 ? 3 * lane + 2 : lane / 2 * 3 + (lane & 1);
  };
  auto wait_slot = [&](int i) -> bool {  // for load i
    return i < kStages || vote(mbar_wait(&bar->kv_empty[i % kStages], (i / kStages - 1) & 1, tmo, abort));
  };
  // K (kv = 0) and V (1) of a segment's tiles, kv0 .. kv1 - 1 of them, into the ring, `before_tile` ahead of
  // each tile; `n` counts the tiles over all segments. A lane's copy of 16 rows takes its warp about 70 ns
  // to issue, and a tile out of 16-row pages is 8 to 16 such copies of K and as many of V, so a helper warp
  // takes a third of both (one warp for K and V held the paged d = 128 cache at 4400 GB/s where a contiguous
  // one ran at 6270). The K and V producers (member 0) announce a tile's bytes; the helper's copies (member
  // 1) may land before that, but the phase waits for the announcement. The helper arrives for every tile, those
  // that hold none of its copies too (drafts, pages of 128 rows, short tails): the ring cannot run on past a load
  // that the helper has not reached, so its waits for slots always mean the use they are for. (Waiting by parity
  // without arriving, two uses behind it took a free slot for a taken one, and its wait ran out at the list's
  // end.)
  auto load_tiles = [&](const Seg& s, int kv0, int kv1, int member, int& n, auto before_tile) -> bool {
    const int nctx = min(max(s.ct - s.k0, 0), s.nt);
    int j = 0;
    if (a.block_table) {
      const int copy = share_copy(member), hfl = copy % C::kHalves, my_piece = (copy / C::kHalves) * a.piece;
      const int* table = a.block_table + static_cast<int64_t>(s.b) * a.max_pages;
      const int pages_on = kKeys / a.page_size, rows_on = kKeys % a.page_size;
      int page, at;
      // the pool row of this lane's piece in the next tile, looked up one tile ahead
      auto pool_row = [&](int kt) -> int {
        if (my_piece >= kKeys || kt >= s.ct || kt * kKeys + my_piece >= s.nk) return -1;
        // a bad entry reads a wrong page, never outside the pool
        return min(max(table[page], 0), a.num_pages - 1) * a.page_size + at;
      };
      // chunks: the tiles that all rows see whole may begin with another than the first; then those before it follow,
      // then the others
      const int turn = kChunk ? s.first : 0, plain = turn > 0 ? min(max(first_masked(s) - s.k0, 0), s.nt) : nctx;
      int kt = s.k0 + turn, run_end = s.k0 + plain;
#pragma unroll 1
      for (int run = 0; run < (turn > 0 ? 3 : 1); ++run) {
        if (run == 1) kt = s.k0, run_end = s.k0 + turn;
        if (run == 2) kt = s.k0 + plain, run_end = s.k0 + nctx;
        // (of a run without tiles, and for a lane without copies, nothing is looked up)
        const int first = kt < s.ct && my_piece < kKeys ? kt * kKeys + my_piece : 0;
        page = first / a.page_size, at = first - page * a.page_size;
        int row_next = pool_row(kt);
#pragma unroll 1
        for (; kt < run_end; ++kt, ++j, ++n) {
          if (!before_tile(j)) return false;
          const int row = row_next;
          page += pages_on;
          if ((at += rows_on) >= a.page_size) at -= a.page_size, ++page;
          row_next = pool_row(kt + 1);
          for (int kv = kv0; kv < kv1; ++kv) {
            const int i = 2 * n + kv, slot = i % kStages;
            if (!wait_slot(i)) {
              // drain() does not know of the K of this tile that went out just before
              if (kv > kv0) mbar_wait(&bar->kv_full[(i - 1) % kStages], ((i - 1) / kStages) & 1, tmo, &no_abort);
              return false;
            }
            if (member == 0) {
              // pieces past the last key are not copied: their K scores are masked, their V rows zeroed
              const int pieces = min(kKeys / a.piece, (s.nk - kt * kKeys + a.piece - 1) / a.piece);
              mbar_arrive_expect_tx(&bar->kv_full[slot], static_cast<uint32_t>(pieces * a.piece) * 128 * C::kHalves);
              __syncwarp();
            }
            if (row >= 0)
              tma_load_3d_lane(sRing + slot * C::kTileBytes + hfl * (kKeys * 128) + my_piece * 128, kv ? &a.tm_v : &a.tm_k,
                               &bar->kv_full[slot], 64 * hfl, s.hkv, row);
            __syncwarp();
            if (member > 0 && lane == 0) mbar_arrive(&bar->kv_full[slot]);
          }
        }
      }
    } else {
#pragma unroll 1
      for (; j < nctx; ++j, ++n) {
        if (!before_tile(j)) return false;
        const int i = 2 * n + kv0, slot = i % kStages;
        if (!wait_slot(i)) return false;
        mbar_arrive_expect_tx(&bar->kv_full[slot], C::kTileBytes);
        for (int hf = 0; hf < C::kHalves; ++hf)
          tma_load_3d(sRing + slot * C::kTileBytes + hf * (kKeys * 128), kv0 ? &a.tm_v : &a.tm_k, &bar->kv_full[slot], 64 * hf,
                      (s.k0 + j) * kKeys, s.b * a.Hkv + s.hkv);
      }
    }
#pragma unroll 1
    for (; !kChunk && j < s.nt; ++j, ++n) {
      if (!before_tile(j)) return false;
      for (int kv = kv0; kv < kv1; ++kv) {
        const int i = 2 * n + kv, slot = i % kStages;
        if (!wait_slot(i)) return false;
        if (member > 0) {  // drafts are the producers' alone
          if (lane == 0) mbar_arrive(&bar->kv_full[slot]);
          __syncwarp();
          continue;
        }
        mbar_arrive_expect_tx(&bar->kv_full[slot], static_cast<uint32_t>(a.new_box) * 128 * C::kHalves);
        for (int hf = 0; hf < C::kHalves; ++hf)
          tma_load_3d(sRing + slot * C::kTileBytes + hf * (kKeys * 128), kv ? &a.tm_vn : &a.tm_kn, &bar->kv_full[slot], 64 * hf,
                      s.hkv, s.tok0 + (s.k0 + j - s.ct) * kKeys);
      }
    }
    return true;
  };
  // the copies a producer warp issued last, of n tiles in all, have landed: those whose slot no later tile took.
  // Where another warp gave up, a slot's phase may never end: the wait that runs out has been the others' time too
  auto drain = [&](int kv, int n) {
    for (int i = 2 * n - 1; i >= max(0, 2 * n - kStages); --i) {
      if ((i & 1) == kv && !mbar_wait(&bar->kv_full[i % kStages], (i / kStages) & 1, tmo, &no_abort)) return;
    }
  };

  if (warp == C::kTmaWarp) {
    // ------------------------------------------------------------ segments, Q and K tiles
    Regs<D, kTiles>::give();
    const int head0 = static_cast<int>(blockIdx.x) - group * a.head_group, end = my_end;
    int pos = my_begin, b = pos < end ? bar->list[1] : 0, seq_at = pos < end ? bar->list[2] : 0;
    int nload = 0, nq[2] = {0, 0};  // K tiles, and Q tiles into each buffer
    // chunks: the sequence (b is the next one), and the unit of it (and of a group of heads) that holds place pos, from place unit_at on
    SeqTiles<D, kTiles, kChunk> seq{};
    int heads = 0, unit = 0, unit_at = 0;
    // Units of a sequence read the same keys, each CTA its run of them. A CTA begins a run with the tile whose number is
    // that of the tiles it has taken, modulo its share: CTAs then read a tile of keys at about the same time, wherever
    // in their units their shares begin, and HBM once for all of them (512 tokens behind 65024, 32/8 heads of 128: 2.15
    // GB of HBM reads in the runs' own order).
    const int share_tiles = max((my_end - my_begin) / P::kTile, 1);
    int taken = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      Seg s{};
      int u0 = 0, size = 0;  // the unit's first place, and its places
      int tile_places = 1;
      while (kChunk && pos < end && !s.valid) {
        for (;;) {
          if (pos >= seq_at + seq.all(a.head_groups)) {  // (before the list's first sequence, seq has no places)
            seq_at += seq.all(a.head_groups);
            seq = seq_tiles<D, kTiles, kChunk>(a, b++);
            seq.count_warp(tile_nodes, lane);
            if (pos >= seq_at + seq.all(a.head_groups)) continue;
            heads = (pos - seq_at) / seq.places;
            unit_at = seq_at + heads * seq.places;
            // its unit, 32 at a time
#pragma unroll 1
            for (unit = 0;; unit += 32) {
              const int n = unit + lane < seq.row_units ? seq.unit_places(unit + lane, tile_nodes) : 0;
              int upto = n;
#pragma unroll
              for (int off = 1; off < 32; off <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, upto, off);
                if (lane >= off) upto += x;
              }
              const unsigned over = __ballot_sync(0xffffffffu, unit_at + upto > pos);
              if (over || unit + 32 >= seq.row_units) {
                const int hit = over ? __ffs(over) - 1 : seq.row_units - 1 - unit;
                unit_at += __shfl_sync(0xffffffffu, upto - n, hit);
                unit += hit;
                break;
              }
              unit_at += __shfl_sync(0xffffffffu, upto, 31);
            }
          }
          tile_places = seq.weight(unit, tile_nodes);
          size = seq.template unit_tiles<kKeys>(unit, kTiles * tile_nodes) * tile_places + P::kCost;
          if (pos < unit_at + size) break;
          unit_at += size;
          if (++unit == seq.row_units) unit = 0, ++heads;
        }
        if (whole_units && pos > unit_at) {  // it began before the range
          pos = unit_at + size;
          continue;
        }
        // the tiles whose first place is in the range
        const int at = pos - unit_at, to = whole_units ? size : min(size, end - unit_at);
        u0 = unit_at;
        pos += to - at;
        s.k0 = (max(at - P::kCost, 0) + tile_places - 1) / tile_places;
        s.nt = (max(to - P::kCost, 0) + tile_places - 1) / tile_places - s.k0;
        if (s.nt <= 0) continue;  // it ends before the unit's first tile, or began inside its last
        s.valid = 1;
        s.b = b - 1;
        s.tok0 = seq.tok0;
        s.nq = seq.nq;
        s.nk = seq.unit_keys(unit, kTiles * tile_nodes);
        s.hkv = heads * a.head_group + head0;
        s.node0 = unit * (kTiles * tile_nodes);
        s.ct = (size - P::kCost) / tile_places;
        s.shift = seq.shift;
        // (a CTA has two parts of units at most: of one that began before its range, and of one that ends behind it)
        s.slot = s.nt == s.ct ? -1 : u0 <= my_begin ? 0 : 1;
        s.split = kTiles == 2 && s.nt > 1 && tile_rows(s, 1) == 0;
        if (seq.row_units > 1) {
          s.first = (taken - s.k0) % share_tiles;
          if (s.first < 0) s.first += share_tiles;
          if (s.first >= min(max(first_masked(s) - s.k0, 0), s.nt)) s.first = 0;
        }
        taken += s.nt;
      }
      while (!kChunk && pos < end && !s.valid) {
        SeqTiles<D, kTiles, kChunk> q = seq_tiles<D, kTiles, kChunk>(a, b);
        while (pos >= seq_at + q.all(a.head_groups)) {
          seq_at += q.all(a.head_groups);
          q = seq_tiles<D, kTiles, kChunk>(a, ++b);
        }
        size = q.per_unit + tree_unit_cost(D);
        const int local = pos - seq_at, unit = local / size;
        const int at = local - unit * size;  // places of the unit
        u0 = pos - at;
        const int to = min(size, end - u0);
        pos += to - at;
        s.k0 = max(at - tree_unit_cost(D), 0);
        s.nt = to - tree_unit_cost(D) - s.k0;
        if (s.nt <= 0) break;  // the range ends before the unit's first tile
        s.valid = 1;
        s.b = b;
        s.tok0 = q.tok0;
        s.nq = q.nq;
        s.nk = q.nk;
        const int heads = q.row_units == 1 ? unit : unit / q.row_units;
        s.hkv = heads * a.head_group + head0;
        s.node0 = (unit - heads * q.row_units) * (kTiles * tile_nodes);
        s.ct = q.ct;
        s.slot = s.nt == q.per_unit ? -1 : (k == 0 ? 0 : 1);
      }
      if (k == 0 && !s.valid && lane == 0) a.merge[blockIdx.x] = TreeMergeRec{};  // no part here
      if (k >= kSegSlots && !(ok = vote(mbar_wait(&bar->seg_empty[k % kSegSlots], (k / kSegSlots - 1) & 1, tmo, abort))))
        break;
      if (lane == 0) {
        bar->seg[k % kSegSlots] = s;
        mbar_arrive(&bar->seg_full[k % kSegSlots]);
      }
      __syncwarp();
      if (!s.valid) break;
      auto load_q = [&]() -> bool {
#pragma unroll
        for (int w = 0; w < kTiles; ++w) {
          if (nq[w] > 0 && !vote(mbar_wait(&bar->q_empty[w], (nq[w] - 1) & 1, tmo, abort))) return false;
          mbar_arrive_expect_tx(&bar->q_full[w], static_cast<uint32_t>(tile_nodes * a.g) * 128 * C::kHalves);
          for (int hf = 0; hf < C::kHalves; ++hf)
            tma_load_3d(sQ + w * C::kQBytes + hf * (kTreeRows * 128) + first_lane * 128, &a.tm_q, &bar->q_full[w], 64 * hf,
                        s.hkv * a.g, s.tok0 + s.node0 + (kChunk && s.split ? 0 : w * tile_nodes));
          ++nq[w];
        }
        return true;
      };
      // later segments: the first loads need ring slots only, not Q's buffer
      const int q_at = k == 0 ? 0 : min(s.nt, (kStages + 3) / 4);
      ok = load_tiles(s, 0, 1, 0, nload, [&](int j) { return j != q_at || load_q(); });
      if (ok && q_at == s.nt) ok = load_q();
      if (k == 0 && lane == 0) {
        // what the merge has to know, once the loads are on their way
        TreeMergeRec r{};
        const Share share(bar->list[0], a.groups, P::kTile);
        if (s.k0 > 0 && share.owner(u0 + P::kCost) == group - 1) {
          r.rows0 = tile_rows(s, 0);
          r.rows1 = kTiles == 2 ? tile_rows(s, 1) : 0;
          r.node0 = s.tok0 + s.node0;
          r.node_step = tile_nodes;
          r.hkv = s.hkv;
          r.slot0 = u0 <= share.begin(group - 1) ? 0 : 1;
          r.last = share.owner(u0 + size - tile_places) * a.head_group + head0;
        }
        a.merge[blockIdx.x] = r;
      }
    }
    if (!ok && lane == 0) raise_timeout(abort, a.status);
    // every copy this warp issued must have landed before the CTA may exit
#pragma unroll
    for (int w = 0; w < kTiles; ++w)
      if (nq[w] > 0) mbar_wait(&bar->q_full[w], (nq[w] - 1) & 1, tmo, &no_abort);
    drain(0, nload);
  } else if (warp >= C::kTmaVWarp) {
    // ------------------------------------------------------------ V tiles, or the helper's share of both
    Regs<D, kTiles>::give();
    const bool helper = warp > C::kTmaVWarp;
    int nload = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const Seg* sp = wait_seg(k);
      if (!(ok = sp != nullptr)) break;
      const Seg s = *sp;
      release_seg(k);
      if (!s.valid) break;
      if (helper && !a.block_table) continue;  // a contiguous cache's tile is kHalves copies
      ok = load_tiles(s, helper ? 0 : 1, 2, helper ? 1 : 0, nload, [](int) { return true; });
    }
    if (!ok && lane == 0) raise_timeout(abort, a.status);
    drain(1, nload);
    if (helper) drain(0, nload);
  } else if (warp >= C::kMmaWarp) {
    // ------------------------------------------------------------ MMA issuers, one per stream
    Regs<D, kTiles>::give();
    const int w = warp - C::kMmaWarp;
    constexpr uint32_t idesc_qk = idesc_bf16_f32(kTreeRows, kKeys, 0, 0);
    constexpr uint32_t idesc_pv = idesc_bf16_f32(kTreeRows, D, 0, 1);
    const uint32_t hi = sdesc_hi(1024);
    const uint32_t q_lo = sdesc_lo(smem_u32(sQ) + (kTiles == 2 ? w : 0) * C::kQBytes, 16);
    const uint32_t k_lo = sdesc_lo(smem_u32(sRing), 16);
    const uint32_t v_lo = sdesc_lo(smem_u32(sRing), kKeys * 128);
    constexpr uint32_t slot_step = C::kTileBytes >> 4;
    const uint32_t tO = tbase + C::kColO + w * D;
    const int qb = kTiles == 2 ? w : 0;
    int nload = 0, ns = 0, np = 0, ou = 0, nturn = 0, nspecial = 0;
    bool ok = true;
    auto wait_load = [&](int i) -> bool {
      const bool r = vote(mbar_wait(&bar->kv_full[i % kStages], (i / kStages) & 1, tmo, abort));
      tc_fence_after();
      return r;
    };
    // S buffer of a stream's n-th tile, and how often the buffer was used before
    auto buf = [&](int n) { return C::kTwoS ? n & 1 : w; };
    auto use = [&](int n) { return C::kTwoS ? n >> 1 : n; };
    // S of load i, whose K has landed
    auto issue_s = [&](int i) {
      const uint32_t kl = k_lo + (i % kStages) * slot_step;
      const uint32_t tS = tbase + C::kColS + buf(ns) * kKeys;
      if constexpr (D == 128) {
        umma_ss_k128(tS, q_lo, hi, kl, hi, idesc_qk, 0);
      } else if constexpr (kQt) {
#pragma unroll
        for (int x = 0; x < 16; ++x)
          umma_ts(tS, tbase + C::kColQ + 8 * x, kl + x / 4 * (kKeys * 128 / 16) + 2 * (x % 4), hi, idesc_qk, x > 0);
      } else {
#pragma unroll
        for (int hf = 0; hf < C::kHalves; ++hf)
          umma_ss_k64(tS, q_lo + hf * (kTreeRows * 128 / 16), hi, kl + hf * (kKeys * 128 / 16), hi, idesc_qk, hf > 0);
      }
      umma_commit(&bar->s_full[buf(ns)]);
      ++ns;
    };
    // the same, once its K has landed and (kSplitP) the softmax has read the previous S
    auto start_s = [&](int i) -> bool {
      if (!wait_load(i)) return false;
      if (C::kSplitP && ns > 0) {
        if (!vote(mbar_wait(&bar->s_free[w], (ns - 1) & 1, tmo, abort))) return false;
        tc_fence_after();
      }
      issue_s(i);
      return true;
    };
    // P.V of load i over the first `valid` keys (whole K = 16 steps)
    auto issue_pv = [&](int i, bool accumulate, int valid, auto special) {
      const uint32_t tP = tbase + (C::kSplitP ? C::kColP + w * 64 : C::kColS + buf(np) * kKeys);
      const uint32_t vl = v_lo + (i % kStages) * slot_step;
      if constexpr (kKeys == 128 && !special) {
        umma_ts_k128(tO, tP, vl, hi, idesc_pv, accumulate ? 1u : 0u);
      } else if constexpr (!special) {
#pragma unroll
        for (int s = 0; s < kKeys / 16; ++s) umma_ts(tO, tP + 8 * s, vl + 128 * s, hi, idesc_pv, (accumulate || s) ? 1u : 0u);
      } else {
#pragma unroll 1
        for (int s = 0; 16 * s < valid; ++s) umma_ts(tO, tP + 8 * s, vl + 128 * s, hi, idesc_pv, (accumulate || s) ? 1u : 0u);
      }
      if constexpr (C::kLook) umma_commit(&bar->pv_done[buf(np)]);
      ++np;
    };
    for (int k = 0; ok; ++k) {
      Seg* sp = wait_seg(k);
      if (!(ok = sp != nullptr)) break;
      const Seg& s = *sp;
      if (!s.valid) {
        release_seg(k);
        break;
      }
      if (!(ok = vote(mbar_wait(kQt ? &bar->qt_full : &bar->q_full[qb], k & 1, tmo, abort)))) break;
      tc_fence_after();
      if (kQt && lane == 0) mbar_arrive(&bar->q_empty[0]);  // copied out of shared memory
      const int nt = s.nt, base = nload;
      nload += 2 * nt;
      // the tiles from `plain` on: the context's last one, if it is not whole, and the drafts
      const int plain = min(max((kChunk ? first_masked(s) : s.nk % kKeys ? s.ct - 1 : s.ct) - s.k0, 0), nt);
      const bool turns = kTiles == 2 && !C::kLook && tile_rows(s, 1) > 0;
      const bool is_split = kChunk && kTiles == 2 && s.split;
      const int j0 = is_split ? w : 0;  // this stream's first tile
      // split: a tile of the other stream's, whose slots are given back once they have been filled
      auto pass_over = [&](int j) -> bool {
        for (int i = base + 2 * j; i < base + 2 * j + 2; ++i) {
          if (!wait_load(i)) return false;
          if (lane == 0) mbar_arrive(&bar->kv_empty[i % kStages]);
          __syncwarp();
        }
        return true;
      };
      if (kTiles == 2 && tile_rows(s, w) == 0 && !is_split) {  // no rows: only gives the slots back
        umma_commit(&bar->q_empty[qb]);
        for (int i = base; ok && i < nload; ++i)
          if ((ok = wait_load(i))) umma_commit(&bar->kv_empty[i % kStages]);
        if (!ok) break;
        nspecial += nt - plain;
        release_seg(k);
        continue;
      }
      if (j0 > 0 && !(ok = pass_over(0))) break;
      if (!(ok = start_s(base + 2 * j0))) break;
      if (!kQt && (is_split ? j0 + 2 >= nt : nt == 1)) umma_commit(&bar->q_empty[qb]);
      // one tile; the special ones are apart, as the issuing warp's time per tile bounds two row tiles
      // (split segments, whose streams take every other tile, too)
      auto tile = [&](int j, auto special, auto split) -> bool {
        constexpr int step = split ? 2 : 1;
        const int ik = base + 2 * j, iv = ik + 1, inext = ik + 2 * step;
        umma_commit(&bar->kv_empty[ik % kStages]);  // S of this tile was issued before
        const bool more = j + step < nt, last_s = j + 2 * step >= nt;
        if (C::kLook && more) {
          // S of the next tile goes ahead of this tile's P.V
          if (!start_s(inext)) return false;
          if (!kQt && last_s) umma_commit(&bar->q_empty[qb]);
        }
        if (!wait_load(iv)) return false;
        int valid = kKeys;  // keys of the tile that count
        if constexpr (special) {
          // P.V stops at the 16 keys that hold the last one that counts; V rows from there to the 16's end
          // are zeroed, and drafts' infinities and NaN (two row tiles read one V tile: stream 0 looks it
          // over for both)
          const int kt = s.k0 + j;
          const bool draft = kChunk ? a.causal != 0 : kt >= s.ct;  // keys that some rows see and others do not
          uint64_t* ready = &bar->v_ready[nspecial % kVSlots];
          valid = min(kKeys, !kChunk && draft ? s.nq - (kt - s.ct) * kKeys : s.nk - kt * kKeys);
          if (kTiles == 1 || w == 0 || split) {
            // (chunks: the keys that the unit's first token sees are seen by all)
            const int from = kChunk ? max(all_see(s) - kt * kKeys, 0) : 0;
            if (clean_v<C::kHalves, kKeys>(sRing + (iv % kStages) * C::kTileBytes, from, valid, draft, lane) && lane == 0)
              atomicOr(&sp->bad, 1);
            __syncwarp();
            if (kTiles == 2 && !split && lane == 0) mbar_arrive(ready);
          } else if (!vote(mbar_wait(ready, (nspecial / kVSlots) & 1, tmo, abort))) {
            return false;
          }
          if (!split) ++nspecial;
        }
        // two row tiles: P.V in turns (0, 1, 0, ...), which keeps the streams out of step, one's softmax
        // beside the other's MMAs
        if (turns) {
          if (w == 1 ? !vote(mbar_wait(&bar->turn[0], nturn & 1, tmo, abort))
                     : nturn > 0 && !vote(mbar_wait(&bar->turn[1], (nturn - 1) & 1, tmo, abort)))
            return false;
        }
        const bool first = split ? j == w : j == 0;
        if (first && ou > 0 && !vote(mbar_wait(&bar->o_empty[w], (ou - 1) & 1, tmo, abort))) return false;
        if (!vote(mbar_wait(&bar->p_full[buf(np)], use(np) & 1, tmo, abort))) return false;
        tc_fence_after();
        issue_pv(iv, !first, valid, special);
        if constexpr (split) {
          umma_commit(&bar->kv_empty[iv % kStages]);
          if (!more) umma_commit(&bar->o_full[w]);
          if (j + 1 < nt && !pass_over(j + 1)) return false;
        }
        if (!more) {
          if (!split) umma_commit(&bar->o_full[w]);
          ++ou;
        } else if (!C::kLook) {
          // S of the next tile overwrites P: it follows this P.V in the warp's stream
          if (!start_s(inext)) return false;
          if (!kQt && last_s) umma_commit(&bar->q_empty[qb]);
        }
        if (turns) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar->turn[w]);
          ++nturn;
        }
        if (!split) umma_commit(&bar->kv_empty[iv % kStages]);
        return true;
      };
      int j = j0;
      if (is_split) {
        if constexpr (kChunk && kTiles == 2) {
#pragma unroll 1
          for (; ok && j < plain; j += 2) ok = tile(j, std::false_type(), std::true_type());
#pragma unroll 1
          for (; ok && j < nt; j += 2) ok = tile(j, std::true_type(), std::true_type());
        }
      } else {
#pragma unroll 1
        for (; ok && j < plain; ++j) ok = tile(j, std::false_type(), std::false_type());
#pragma unroll 1
        for (; ok && j < nt; ++j) ok = tile(j, std::true_type(), std::false_type());
      }
      if (!ok) break;
      release_seg(k);
    }
    if (!ok && lane == 0) raise_timeout(abort, a.status);
    // all MMAs issued by this warp complete before TMEM is released
    umma_commit(&bar->mma_done[w]);
    mbar_wait(&bar->mma_done[w], 0, tmo, &no_abort);
  } else {
    // ------------------------------------------------------------ softmax warpgroups
    Regs<D, kTiles>::take();
    const int w = warp >> 2;
    const int row = (warp & 3) * 32 + lane - first_lane;  // of the tile: the TMEM lane less that of the first row
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tO = tbase + lane_base + C::kColO + w * D;
    const float sl2 = a.scale_log2;
    int n = 0, oused = 0, nsplit = 0;
    bool ok = true;
    // Q of the k-th segment from shared memory (128-byte swizzle) into tensor memory, a thread's row each; every S of the
    // segment before is complete
    auto copy_q = [&](int k) -> bool {
      if (!vote(mbar_wait(&bar->q_full[0], k & 1, tmo, abort))) return false;
      const int r = (warp & 3) * 32 + lane;
#pragma unroll 1
      for (int hf = 0; hf < C::kHalves; ++hf) {
        uint32_t v[32];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 x = *reinterpret_cast<const uint4*>(sQ + hf * (kTreeRows * 128) + r * 128 + ((c ^ (r & 7)) << 4));
          v[4 * c] = x.x, v[4 * c + 1] = x.y, v[4 * c + 2] = x.z, v[4 * c + 3] = x.w;
        }
        tmem_st32(tbase + lane_base + C::kColQ + 32 * hf, v);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&bar->qt_full);
      return true;
    };
    for (int k = 0; ok; ++k) {
      const Seg* sp = wait_seg(k);
      if (!(ok = sp != nullptr)) break;
      const Seg s = *sp;
      if (!s.valid) {
        release_seg(k);
        break;
      }
      if (kQt && k == 0 && !(ok = copy_q(0))) break;
      const bool is_split = kChunk && kTiles == 2 && s.split;
      const int rw = kTiles == 2 && !is_split ? w : 0;        // row tile of this stream
      const int rows = tile_rows(s, rw);
      if (rows == 0) {
        release_seg(k);
        continue;
      }
      const bool row_ok = row >= 0 && row < rows, warp_ok = row - lane >= 0 && row - lane < rows;
      const int some_row = min(max(row, 0), rows - 1);
      const int node = s.node0 + rw * tile_nodes + some_row / a.g;  // within the sequence
      const int head = s.hkv * a.g + some_row % a.g;
      const uint64_t* bits = kChunk ? nullptr : a.mask + static_cast<int64_t>(s.tok0 + node) * a.mask_words;
      const int limit = kChunk ? min(max(s.shift + node + 1, 0), s.nk) : 0;  // keys that this row sees
      // the tiles from `plain` on have keys that some row does not see
      const int plain = min(max((kChunk ? first_masked(s) : s.nk % kKeys ? s.ct - 1 : s.ct) - s.k0, 0), s.nt);
      float m_ref = -INFINITY, l = 0.f;
      // (split segments: j counts the stream's own tiles, every other one. Their loops are apart, as the common ones take
      // up to 5 % longer with a choice inside)
      auto tile = [&](int j, auto masked, auto split) -> bool {
        const int x = C::kTwoS ? n & 1 : w, phase = (C::kTwoS ? n >> 1 : n) & 1;
        const uint32_t tS = tbase + lane_base + C::kColS + x * kKeys;
        const uint32_t tP = C::kSplitP ? tbase + lane_base + C::kColP + w * 64 : tS;
        if (!vote(mbar_wait(&bar->s_full[x], phase, tmo, abort))) return false;
        tc_fence_after();
        if (warp_ok) {
          float alpha_o = 1.f;
          if constexpr (masked) {
            const int kt = s.k0 + (split ? 2 * j + w : j);
            if (C::kSplitP && n > 0) {
              if (!vote(mbar_wait(&bar->pv_done[x], (n - 1) & 1, tmo, abort))) return false;
              tc_fence_after();
            }
            const bool draft = !kChunk && kt >= s.ct;
            const int left = draft ? s.nq - (kt - s.ct) * kKeys : s.nk - kt * kKeys;
            const MaskedTile r = masked_tile<kChunk>(tS, tP, min(left, kKeys), limit - kt * kKeys, draft ? bits : nullptr,
                                                     (kt - s.ct) * kKeys, sl2, m_ref);
            m_ref = r.m;
            l = l * r.alpha + r.l;
            if (j > 0) alpha_o = r.alpha;
            if constexpr (C::kSplitP) {
              tc_fence_before();
              mbar_arrive(&bar->s_free[x]);
            }
          } else {
            uint32_t sc[kKeys / 32][32];
#pragma unroll
            for (int c = 0; c < kKeys / 32; ++c) tmem_ld32(tS + 32 * c, sc[c]);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < kKeys / 32; ++c) tmem_reg_fence(sc[c]);
            if constexpr (C::kSplitP) {
              tc_fence_before();
              mbar_arrive(&bar->s_free[x]);  // S is in registers
            }
            float mx[kKeys / 32];
#pragma unroll
            for (int c = 0; c < kKeys / 32; ++c) {
              mx[c] = __uint_as_float(sc[c][0]);
#pragma unroll
              for (int e = 1; e < 31; e += 2) mx[c] = max3f(mx[c], __uint_as_float(sc[c][e]), __uint_as_float(sc[c][e + 1]));
              mx[c] = fmaxf(mx[c], __uint_as_float(sc[c][31]));
            }
            float mt = mx[0];
#pragma unroll
            for (int c = 1; c < kKeys / 32; ++c) mt = fmaxf(mt, mx[c]);
            const float m_new = fmaxf(m_ref, mt * sl2);
            if (m_new > m_ref + kRescaleThreshold) {
              const float alpha = (m_ref == -INFINITY) ? 0.f : ex2(m_ref - m_new);
              l *= alpha;
              if (j > 0) alpha_o = alpha;
              m_ref = m_new;
            }
            const float nm = (m_ref == -INFINITY) ? 0.f : -m_ref;
            if (C::kSplitP && n > 0) {
              // the stream's previous P.V has read the P columns, and O holds it
              if (!vote(mbar_wait(&bar->pv_done[x], (n - 1) & 1, tmo, abort))) return false;
              tc_fence_after();
            }
            // p = 2^(s scale log2e - m) as bf16 pairs into the first half of the S columns. The tensor core
            // multiplies bf16 V by weights of the same type only: each is off by at most 2^-8 of itself, the
            // output type's own half step (measured on the listed sizes, 2.3e-3 from 64 bits, fp32 weights
            // rounded once at the end 1.7e-3). l is the fp32 sum before that rounding
            float ls[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < kKeys / 32; ++c) {
              uint32_t pk[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                float x0, x1;
                ffma2(x0, x1, __uint_as_float(sc[c][2 * e]), __uint_as_float(sc[c][2 * e + 1]), sl2, nm);
                const float p0 = ex2(x0), p1 = ex2(x1);
                fadd2(ls[(2 * e) & 7], ls[(2 * e + 1) & 7], p0, p1);
                pk[e] = pack_bf16x2(p0, p1);
              }
              tmem_st16(tP + 16 * c, pk);
            }
            l += ((ls[0] + ls[1]) + (ls[2] + ls[3])) + ((ls[4] + ls[5]) + (ls[6] + ls[7]));
          }
          // O must carry the new reference maximum before this tile's P.V (rare)
          if (__any_sync(0xffffffffu, alpha_o != 1.f)) {
            if (C::kTwoS) {
              // S(j) was issued ahead of P.V(j - 1): that one has to be done
              if (!vote(mbar_wait(&bar->pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1, tmo, abort))) return false;
              tc_fence_after();
            }
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t ov[32];
              tmem_ld32(tO + c * 32, ov);
              tmem_wait_ld();
              tmem_reg_fence(ov);
#pragma unroll
              for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha_o);
              tmem_st32(tO + c * 32, ov);
            }
          }
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&bar->p_full[x]);
        } else {
          if constexpr (C::kSplitP) {
            // a warp without rows may not run ahead either: its arrivals for the next P would count for this
            mbar_arrive(&bar->s_free[x]);
            if (n > 0 && !vote(mbar_wait(&bar->pv_done[x], (n - 1) & 1, tmo, abort))) return false;
          }
          mbar_arrive(&bar->p_full[x]);
        }
        ++n;
        return true;
      };
      auto loops = [&](int masked_from, int end, auto split) {
        int j = 0;
#pragma unroll 1
        for (; ok && j < masked_from; ++j) ok = tile(j, std::false_type(), split);
#pragma unroll 1
        for (; ok && j < end; ++j) ok = tile(j, std::true_type(), split);
      };
      if (is_split) {
        if constexpr (kChunk && kTiles == 2) loops((plain + 1 - w) / 2, (s.nt + 1 - w) / 2, std::true_type());
      } else {
        loops(plain, s.nt, std::false_type());
      }
      if (!ok) break;
      if constexpr (kQt) {
        // the next segment's first scores are computed while this one's end is written
        const Seg* next = wait_seg(k + 1);
        if (!(ok = next != nullptr) || (next->valid && !(ok = copy_q(k + 1)))) break;
      }
      // ---- the unit's end in this CTA
      if (!(ok = vote(mbar_wait(&bar->o_full[w], oused & 1, tmo, abort)))) break;
      ++oused;
      tc_fence_after();
      float f0 = 1.f, f1 = 0.f;  // split: the streams' shares of O
      if (is_split) {
        // the streams' parts are joined here: stream 0 takes stream 1's O from tensor memory, lane for lane. (What
        // stream 1 writes for the next split segment comes behind that one's P.V, which waits for o_empty.)
        float2* ml = reinterpret_cast<float2*>(smem + C::kMl) + ((warp & 3) * 32 + lane);
        if (w == 1) {
          *ml = make_float2(m_ref, l);
          tc_fence_before();
          mbar_arrive(&bar->ml_full);
          release_seg(k);
          continue;
        }
        if (!(ok = vote(mbar_wait(&bar->ml_full, nsplit & 1, tmo, abort)))) break;
        ++nsplit;
        tc_fence_after();
        const float2 other = *ml;
        const float m = fmaxf(m_ref, other.x);
        f0 = m_ref == -INFINITY ? 0.f : ex2(m_ref - m);
        f1 = other.x == -INFINITY ? 0.f : ex2(other.x - m);
        l = l * f0 + other.y * f1;
        m_ref = m;
      }
      if (warp_ok) {
        const bool bad = *const_cast<const volatile int*>(&sp->bad) != 0;
        const int64_t orow = static_cast<int64_t>(s.tok0 + node) * a.Hq + head;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        float* part = a.partial + ((static_cast<int64_t>(blockIdx.x) * 2 + max(s.slot, 0)) * kTiles + rw) * (kTreeRows * (D + 2));
        if (kChunk && s.slot < 0 && !bad && !is_split && s.nk > 0) {
          write_rows<D>(tO, inv, row_ok ? orow : -1, a.o, lane);
        } else {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t ov[32];
            tmem_ld32(tO + c * 32, ov);
            tmem_wait_ld();
            tmem_reg_fence(ov);
            float o[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(ov[e]);
            if constexpr (kChunk && kTiles == 2) {
              if (is_split) {
                tmem_ld32(tO + D + c * 32, ov);
                tmem_wait_ld();
                tmem_reg_fence(ov);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = o[e] * f0 + __uint_as_float(ov[e]) * f1;
              }
            }
            if (bad && row_ok) {
              // the infinities and NaN among the drafts (chunks: among the keys of masked tiles) that this row sees
              if constexpr (kChunk) {
                const int* table = a.block_table + static_cast<int64_t>(s.b) * a.max_pages;
                // (the end of the last tile may be 2^31: tables hold up to 2^31 - 1 keys)
                const int d1 = static_cast<int>(min(static_cast<int64_t>(s.k0 + s.nt) * kKeys, static_cast<int64_t>(limit)));
                for (int x = max(s.k0 * kKeys, all_see(s)); x < d1; ++x) {
                  const int page = min(max(table[x / a.page_size], 0), a.num_pages - 1);
                  const uint16_t* v = a.v + ((static_cast<int64_t>(page) * a.page_size + x % a.page_size) * a.Hkv + s.hkv) * D + c * 32;
#pragma unroll
                  for (int e = 0; e < 32; ++e)
                    if ((v[e] & 0x7f80) == 0x7f80) o[e] += __uint_as_float(static_cast<uint32_t>(v[e]) << 16);
                }
              }
              const int d0 = max(s.k0 - s.ct, 0) * kKeys, d1 = min((s.k0 + s.nt - s.ct) * kKeys, s.nq);
              for (int x = d0; !kChunk && x < d1; ++x) {
                if (!(bits[x >> 6] >> (x & 63) & 1)) continue;
                const uint16_t* v = a.v_new + (s.tok0 + x) * a.v_new_stride + s.hkv * D + c * 32;
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if ((v[e] & 0x7f80) == 0x7f80) o[e] += __uint_as_float(static_cast<uint32_t>(v[e]) << 16);
              }
            }
            if constexpr (kChunk) {
              // a unit without keys has no P.V: what stands in tensor memory is not its O
              if (s.nk == 0)
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = 0.f;
            }
            if (!row_ok) continue;
            if (s.slot < 0) {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                uint4 v;
                v.x = pack_bf16x2(o[8 * q] * inv, o[8 * q + 1] * inv);
                v.y = pack_bf16x2(o[8 * q + 2] * inv, o[8 * q + 3] * inv);
                v.z = pack_bf16x2(o[8 * q + 4] * inv, o[8 * q + 5] * inv);
                v.w = pack_bf16x2(o[8 * q + 6] * inv, o[8 * q + 7] * inv);
                *reinterpret_cast<uint4*>(a.o + orow * D + c * 32 + 8 * q) = v;
              }
            } else {
#pragma unroll
              for (int q = 0; q < 8; ++q)
                *reinterpret_cast<float4*>(part + ((c * 8 + q) * kTreeRows + row) * 4) =
                    make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
            }
          }
        }
        if (row_ok && s.slot < 0 && a.lse) a.lse[orow] = l == 0.f ? -INFINITY : (m_ref + log2f(l)) * kLn2;
        if (row_ok && s.slot >= 0) *reinterpret_cast<float2*>(part + kTreeRows * D + 2 * row) = make_float2(m_ref, l);
      }
      tc_fence_before();
      mbar_arrive(&bar->o_empty[w]);
      if (is_split) mbar_arrive(&bar->o_empty[1]);
      release_seg(k);
    }
    if (!ok && lane == 0) raise_timeout(abort, a.status);
    tc_fence_before();
  }
  __syncthreads();
  if (warp == C::kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tbase, C::kCols);
  }
}

// The parts of units that several CTAs shared. At most one unit per boundary between two CTAs has to
// be merged, so the grid is (boundaries, quarters of a row tile x row tiles, groups of 32 channels),
// whatever the lengths; or, where the call has fewer units than that, (units, ...), each block counting
// its way to its record (2 x 8 units of 8192 keys on 304 CTAs: 21.5 us in all, with a block for every
// boundary, most of them empty, 24.4; one warp a block reads the records, as all eight made their few lines
// of L2 a bottleneck and took 4 us). Lanes are rows; the warps (as many as a unit has parts on average, up to
// kMergeWarps) share out the parts, each with its own running maximum, and are joined in shared memory in
// their order:
//   m = max m_c, l = sum l_c 2^(m_c - m), o likewise.
// What bounds it is latency: the records, then the parts. So a warp has two parts' loads under way (the parts
// of 8 units of 4096 keys on 280 CTAs: 14.8 us in all, one at a time 16.6).
constexpr int kMergeWarps = 8;
constexpr int kMergeQuads = 8;  // channels of a block, in fours
constexpr uint32_t merge_smem(int warps) { return warps * (kMergeQuads * 33 * 16 + 32 * 8); }
__global__ void __launch_bounds__(kMergeWarps * 32)
    tree_merge_kernel(const float* partial, const TreeMergeRec* merge, uint16_t* out, float* lse, int D, int quarters, int tiles, int g,
                      int Hq, int head_group, int ctas) {
  const int warps = blockDim.x / 32;
  extern __shared__ float4 sm_merge[];
  auto sm_o = reinterpret_cast<float4 (*)[kMergeQuads][33]>(sm_merge);  // 33: the joining threads' columns fall on different banks
  auto sm_ml = reinterpret_cast<float2 (*)[32]>(sm_merge + warps * kMergeQuads * 33);
  __shared__ int sm_c;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the parts and records are complete and visible
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int c = blockIdx.x + head_group;
  if (head_group + static_cast<int>(gridDim.x) < ctas) {
    if (warp == 0) {
      // the blockIdx.x-th record with rows: lane i holds those of records 32 i .. 32 i + 31 as bits
      constexpr int kWords = (kTreeMaxCtas + 31) / 32;
      int rows[kWords];
#pragma unroll
      for (int i = 0; i < kWords; ++i)
        rows[i] = head_group + 32 * i + lane < ctas ? __ldcg(&merge[head_group + 32 * i + lane].rows0) : 0;
      unsigned some = 0;
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const unsigned bits = __ballot_sync(0xffffffffu, rows[i] > 0);
        if (lane == i) some = bits;
      }
      int upto = __popc(some);
#pragma unroll
      for (int off = 1; off < kWords; off <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += x;
      }
      int left = blockIdx.x - (upto - __popc(some));  // of this lane's bits
      if (left >= 0 && left < __popc(some)) {
        for (; left > 0; --left) some &= some - 1;
        sm_c = head_group + 32 * lane + __ffs(some) - 1;
      }
      if (lane == kWords - 1 && upto <= static_cast<int>(blockIdx.x)) sm_c = 0;  // no such record
    }
    __syncthreads();
    c = sm_c;
    if (c == 0) return;
  }
  const int w = static_cast<int>(blockIdx.y) / quarters, quarter = static_cast<int>(blockIdx.y) - w * quarters, cg = blockIdx.z;
  const int4 r0 = __ldcg(reinterpret_cast<const int4*>(merge + c)), r1 = __ldcg(reinterpret_cast<const int4*>(merge + c) + 1);
  const int rows = w ? r0.y : r0.x, hkv = r1.x, slot0 = r1.y, last = r1.z;
  if (32 * quarter >= rows) return;
  const int row = 32 * quarter + lane;
  float m = -INFINITY, l = 0.f;
  float4 acc[kMergeQuads];
#pragma unroll
  for (int q = 0; q < kMergeQuads; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (row < rows) {
    struct Part {
      float2 ml;
      float4 v[kMergeQuads];
    };
    auto load = [&](int x, Part& part) {
      const float* p = partial + ((static_cast<int64_t>(x) * 2 + (x < c ? slot0 : 0)) * tiles + w) * (kTreeRows * (D + 2));
      part.ml = __ldcg(reinterpret_cast<const float2*>(p + kTreeRows * D + 2 * row));
#pragma unroll
      for (int q = 0; q < kMergeQuads; ++q)
        part.v[q] = __ldcg(reinterpret_cast<const float4*>(p + ((cg * kMergeQuads + q) * kTreeRows + row) * 4));
    };
    const int step = warps * head_group;
#pragma unroll 1
    for (int x = c + (warp - 1) * head_group; x <= last; x += 2 * step) {
      // two parts' loads at a time: the loop is as long as their latency
      Part a, b;
      load(x, a);
      if (x + step <= last) {
        load(x + step, b);
      } else {
        b.ml = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int q = 0; q < kMergeQuads; ++q) b.v[q] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      const float mn = max3f(m, a.ml.x, b.ml.x);
      const float f0 = m == -INFINITY ? 0.f : ex2(m - mn), f1 = a.ml.x == -INFINITY ? 0.f : ex2(a.ml.x - mn),
                  f2 = b.ml.x == -INFINITY ? 0.f : ex2(b.ml.x - mn);
      m = mn;
      l = l * f0 + a.ml.y * f1 + b.ml.y * f2;
#pragma unroll
      for (int q = 0; q < kMergeQuads; ++q) {
        acc[q].x = acc[q].x * f0 + a.v[q].x * f1 + b.v[q].x * f2;
        acc[q].y = acc[q].y * f0 + a.v[q].y * f1 + b.v[q].y * f2;
        acc[q].z = acc[q].z * f0 + a.v[q].z * f1 + b.v[q].z * f2;
        acc[q].w = acc[q].w * f0 + a.v[q].w * f1 + b.v[q].w * f2;
      }
    }
  }
  sm_ml[warp][lane] = make_float2(m, l);
#pragma unroll
  for (int q = 0; q < kMergeQuads; ++q) sm_o[warp][q][lane] = acc[q];
  __syncthreads();
  const int used = min(warps, (last - c) / head_group + 2);
  for (int i = threadIdx.x; i < 32 * kMergeQuads; i += blockDim.x) {
    const int jr = i / kMergeQuads, jq = i % kMergeQuads;  // row, channel quad
    const int rr = 32 * quarter + jr;
    if (rr >= rows) break;
    float M = -INFINITY, L = 0.f;
    for (int x = 0; x < used; ++x) M = fmaxf(M, sm_ml[x][jr].x);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x = 0; x < used; ++x) {
      const float2 ml = sm_ml[x][jr];
      const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
      const float4 v = sm_o[x][jq][jr];
      L += ml.y * f;
      o.x += v.x * f;
      o.y += v.y * f;
      o.z += v.z * f;
      o.w += v.w * f;
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const int64_t orow = static_cast<int64_t>(r0.z + w * r0.w + rr / g) * Hq + hkv * g + rr % g;
    *reinterpret_cast<uint2*>(out + orow * D + 4 * (cg * kMergeQuads + jq)) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (lse && cg == 0 && jq == 0) lse[orow] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
  }
}

template <int D, int kTiles, bool kChunk>
cudaError_t launch(const TreeArgs& a, int dev, cudaStream_t stream) {
  using C = Cfg<D, kTiles>;
  // once per device (the attribute stays with the device's copy of the kernel)
  static std::atomic<uint64_t> set{0};
  cudaError_t e;
  if (dev >= 64 || !(set.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(tree_kernel<D, kTiles, kChunk>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::kSmem));
    if (e != cudaSuccess) return e;
    if (dev < 64) set.fetch_or(1ull << dev);
  }
  e = launch_dependent(tree_kernel<D, kTiles, kChunk>, dim3(a.groups * a.head_group), C::kThreads, C::kSmem, stream, a);
  if (e != cudaSuccess) return e;
  count_launch();
  if (a.groups == 1) return cudaSuccess;
  const int quarters = a.tile_rows / 32;
  e = launch_dependent(tree_merge_kernel, dim3(a.merges, quarters * kTiles, D / (4 * kMergeQuads)), a.merge_warps * 32,
                       merge_smem(a.merge_warps), stream, a.partial, a.merge, a.o, a.lse, D, quarters, kTiles, a.g, a.Hq,
                       a.head_group, a.groups * a.head_group);
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace

cudaError_t launch_tree(TreeArgs& a, void* workspace, cudaStream_t stream) {
  cudaError_t e = status_word(&a.status);
  if (e != cudaSuccess) return e;
  a.timeout_ns = wait_timeout_ns();
  a.merge = static_cast<TreeMergeRec*>(workspace);
  a.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kTreeMergeBytes);
  const int d = a.d, keys = d == 256 ? 64 : 128;
  a.tile_rows = tree_tile_rows(a.max_nodes, a.g, d);
  a.tile_nodes = a.tile_rows / a.g;
  if ((e = make_map_bf16(&a.tm_q, a.q, d, a.Hq, a.total_q, d, a.q_stride, a.g, a.tile_nodes)) != cudaSuccess) return e;
  const bool chunk = a.k_new == nullptr;
  a.new_box = a.max_nodes < keys ? (a.max_nodes + 7) / 8 * 8 : keys;
  if (!chunk && ((e = make_map_bf16(&a.tm_kn, a.k_new, d, a.Hkv, a.total_q, d, a.k_new_stride, 1, a.new_box)) != cudaSuccess ||
                 (e = make_map_bf16(&a.tm_vn, a.v_new, d, a.Hkv, a.total_q, d, a.v_new_stride, 1, a.new_box)) != cudaSuccess))
    return e;
  if (a.kv_cap == 0) {
    a.tm_k = a.tm_kn;  // no context tile exists
    a.tm_v = a.tm_vn;
  } else if (a.block_table) {
    a.piece = 16;
    while (a.piece < keys && a.page_size % (2 * a.piece) == 0) a.piece *= 2;
    const int64_t rows = static_cast<int64_t>(a.num_pages) * a.page_size, step = static_cast<int64_t>(a.Hkv) * d;
    if ((e = make_map_bf16(&a.tm_k, a.k, d, a.Hkv, rows, d, step, 1, a.piece)) != cudaSuccess ||
        (e = make_map_bf16(&a.tm_v, a.v, d, a.Hkv, rows, d, step, 1, a.piece)) != cudaSuccess)
      return e;
  } else {
    const int64_t heads = static_cast<int64_t>(a.num_seqs) * a.Hkv, step = static_cast<int64_t>(a.kv_cap) * d;
    if ((e = make_map_bf16(&a.tm_k, a.k, d, a.kv_cap, heads, d, step, keys, 1)) != cudaSuccess ||
        (e = make_map_bf16(&a.tm_v, a.v, d, a.kv_cap, heads, d, step, keys, 1)) != cudaSuccess)
      return e;
  }
  int dev = 0, sms = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  const int tiles = tree_row_tiles(a.max_nodes, a.g, d);
  const int64_t most = tree_most_tiles(a);  // no more CTAs than tiles there can be
  const int fit = tiles == 1 && d <= 128 ? 2 * sms : sms;
  const int ctas = tree_max_ctas(tiles, d) < fit ? tree_max_ctas(tiles, d) : fit;
  // a page holds the rows of all KV heads side by side: CTAs that read the same keys of different heads at
  // the same time share the pages of HBM that these lie in (16 x 32768 keys, d = 64, 16-token pages: 179 us,
  // each head on its own 202)
  a.head_group = a.block_table ? tree_head_group(a.Hkv, ctas) : 1;
  a.head_groups = a.Hkv / a.head_group;
  a.groups = ctas / a.head_group;
  if (a.groups > most / a.head_group) a.groups = static_cast<int>(most / a.head_group);
  const int64_t boundaries = static_cast<int64_t>(a.groups - 1) * a.head_group, units = tree_most_units(a);
  a.merges = static_cast<int>(units < boundaries ? units : boundaries);
  a.merge_warps = kMergeWarps;  // a power of two, at least the parts of a unit on average
  while (a.merge_warps > 2 && boundaries / units + 2 <= a.merge_warps / 2) a.merge_warps /= 2;
  auto go = [&](auto is_chunk) {
    constexpr bool kChunk = decltype(is_chunk)::value;
    if (d == 64) return tiles == 2 ? launch<64, 2, kChunk>(a, dev, stream) : launch<64, 1, kChunk>(a, dev, stream);
    if (d == 128) return tiles == 2 ? launch<128, 2, kChunk>(a, dev, stream) : launch<128, 1, kChunk>(a, dev, stream);
    return launch<256, 1, kChunk>(a, dev, stream);
  };
  return chunk ? go(std::true_type()) : go(std::false_type());
}

}  // namespace bw
