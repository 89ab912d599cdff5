// Norm and rotation of queries and keys in one pass, rows of a projection in, q and k for attention out:
//   n_c = x_c w_c / sqrt(mean x^2 + eps)            (a head's d channels; without a weight n = x)
//   (a, b) -> (a cos t - b sin t, a sin t + b cos t)  for each pair of channels, t = position * frequency,
// pairs (c, c + pairs) or, interleaved, (2 c, 2 c + 1); the position comes from the pair's axis (time, height,
// width). Channels behind the pairs are normalised only. 32 bits in between, rounded to bf16 once.
//
// What bounds it: every value is read and written once, 4 bytes each, and few instructions may be spent on them.
// A warp takes whole rows, some heads a turn: d / 16 lanes a head, each with two pieces of 8 channels that hold both
// halves of its pairs, so rotating needs no exchange. Weights, cosines and sines are multiplied once a row: an
// output is r (x C + other S), with r the head's 1 / sqrt and `other` the pair's other channel, in packed pairs of
// 32 bits. The coming turns' values are copied to shared memory meanwhile. 16384 rows of 32 + 8 heads of 128: 54.4 us,
// 6.2 TB/s, with neighbours as pairs 54.3, without norms 54.2, in place 55.5 (weights and rotation apart, in single
// values: 78 us and 2400 instructions a row; a row shared by a block's warps, with a barrier a row: 59.6; five blocks an
// SM in 96 registers: 61.4). Of 64 channels 28.8 us for half the bytes, 16 + 4 heads of 256 59.5; 32 pairs of 128 channels 65.3.
#include <math.h>

#include <type_traits>

#include "kernels.h"
#include "packed.cuh"
#include "ptx.cuh"

namespace bw {

namespace {

constexpr int kRopeThreads = 128;

enum RopeMode { kHalves, kAdjacent, kHalvesAny };  // kHalvesAny: pairs no multiple of 8

// A rotation's angle in turns is position * frequency / 2 pi modulo 1: with frequency / 2 pi as a fraction of 2^64
// the product of integers wraps to just that, however far the position. The frequency's 24 bits times 1 / 2 pi
// in 2^-64ths (cut off: at most 2^-61 of itself), exactly, shifted by its exponent, which cuts off at most 2^-64 of a turn
// (2^-63 next to a whole one, see kNoTurn). A frequency of 1 at position 2^31 is so off by 2^-32 of a turn, as much as
// cos_sin() cuts off.
// Infinities and NaN have no angle: kNoTurn, for which the smallest turns of either sign, 2^-64, give way to twice that.
constexpr uint64_t kNoTurn = 1;
__device__ __forceinline__ uint64_t turn_of(float freq) {
  constexpr uint64_t kInvTwoPi = 0x28be60db9391054aull;  // 1 / 2 pi, in 2^-64ths
  const uint32_t bits = __float_as_uint(freq), e = bits >> 23 & 255;
  const uint64_t m = e ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
  const int down = 150 - static_cast<int>(e ? e : 1);  // freq = m 2^-down
  const uint64_t lo = m * kInvTwoPi, hi = __umul64hi(m, kInvTwoPi);
  uint64_t t;
  if (down <= 0)
    t = -down < 64 ? lo << -down : 0;
  else if (down < 64)
    t = lo >> down | hi << (64 - down);
  else
    t = down < 128 ? hi >> (down - 64) : 0;
  if (e == 255) return kNoTurn;
  if (t == kNoTurn) t = 2;
  if (t == 0 - kNoTurn) t = 0 - 2ull;
  return bits >> 31 ? 0 - t : t;
}
__device__ __forceinline__ float2 cos_sin(int position, uint64_t turn) {
  const uint64_t x = static_cast<uint64_t>(static_cast<int64_t>(position)) * turn;
  float s, c;
  sincospif(static_cast<float>(static_cast<int32_t>(x >> 32)) * 0x1p-31f, &s, &c);
  return turn == kNoTurn ? make_float2(NAN, NAN) : make_float2(c, s);
}

__device__ __forceinline__ pair_t unpack(uint32_t w) { return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
__device__ __forceinline__ uint32_t pack(pair_t x) { return pack_bf16x2(first(x), second(x)); }
__device__ __forceinline__ float bf16(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }

// A head's 1 / sqrt is of its sum of squares, which may pass 2^128, or vanish where eps does not hide that (a mean square
// loses 2^-126 at most, which counts below 2^-100). Such a head's squares are taken once more, of values 2^-96 or 2^96 times
// as large, which lie between 2^-37 and 2^51 where they count. An eps below 2^-100 has its own instances (kTiny), as what
// the small values need there costs the others up to 5 % (16384 rows of 32 + 8 heads of 128: 57.2 us; the check for the
// large ones 0.3, where every head of q is one 77 in all; 16 + 4 heads of 256 58.3 without it).
constexpr float kTinyEps = 0x1p-100f;

// A warp takes a row's heads (or one of `gridDim.y` parts of them), kHeads a turn, and then another row's.
constexpr int kRing = 3;        // turns that a warp has under way (16384 rows of 32 + 8 heads of 128: 54.3 us, 4 54.9, 6 57.1)
constexpr int kRopeBlocks = 4;  // an SM

template <int D, int kMode, bool kTiny>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks) qk_rope_kernel(const RopeArgs a, int per_part) {
  constexpr int kLanes = D / 16, kHeads = 32 / kLanes;  // lanes a head, heads a turn
  constexpr int kWarps = kRopeThreads / 32, kMine = D / 64;  // kMine: a lane's pairs
  __shared__ __align__(16) float sm_coef[kWarps][2][2][D];  // C and S of q's channels and of k's
  // kHalvesAny: a turn's values; a word between pieces and some between heads, so that a warp's lanes, each at the same
  // place of its piece, are in 32 banks (16384 rows of 40 heads of 128, 17 pairs: without them 101 us, with them, and
  // second pieces left alone where they hold no pair, 79)
  constexpr int kHeadWords = D + D / 8 + (D == 64 ? 28 : D == 128 ? 24 : 16);
  static_assert(kHeadWords % 32 == 9 * kLanes % 32, "banks");
  __shared__ float sm_x[kMode == kHalvesAny ? kWarps : 1][kMode == kHalvesAny ? kHeads : 1][kMode == kHalvesAny ? kHeadWords : 1];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t = lane % kLanes, group = lane / kLanes;
  // turns: of q's heads first, then of k's; the part's
  const int q_turns = (a.Hq + kHeads - 1) / kHeads, turns = q_turns + (a.Hkv + kHeads - 1) / kHeads;
  const int turn0 = static_cast<int>(blockIdx.y) * per_part, turn1 = min(turn0 + per_part, turns);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  if (row >= a.num_rows) return;
  // the two pieces: both halves of 8 pairs, or neighbours among the channels that are not turned
  const int half = a.pairs / 8;
  const bool turned = kMode != kHalves || t < half;
  const int pa = turned ? t : 2 * t, pb = kMode != kHalves ? t + kLanes : turned ? t + half : 2 * t + 1;
  // The coming turns' values are copied to shared memory, over the ends of rows; a lane reads what it copied itself.
  extern __shared__ uint4 sm_raw[];
  uint4* ring = sm_raw + warp * (kRing * 64) + lane;
  int64_t f_row = row;
  int f_turn = turn0, f_slot = 0;
  auto fetch = [&]() {
    const bool is_k = f_turn >= q_turns;
    const int head = (is_k ? f_turn - q_turns : f_turn) * kHeads + group;
    if (f_row < a.num_rows && head < (is_k ? a.Hkv : a.Hq)) {
      const uint4* src = reinterpret_cast<const uint4*>((is_k ? a.k + f_row * a.k_stride : a.q + f_row * a.q_stride) + head * D);
      uint4* dst = ring + f_slot * 64;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src + pa) : "memory");
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst + 32)), "l"(src + pb) : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    f_slot = f_slot + 1 == kRing ? 0 : f_slot + 1;
    if (++f_turn == turn1) f_turn = turn0, f_row += step;
  };
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) fetch();
  // a lane's pairs: their channels, the channels' weights, the turns a position, the next row's position
  int axis_row[kMine] = {}, pos[kMine];
  uint64_t my_turn[kMine];
  auto position = [&](int i, int64_t r) {
    return 32 * i + lane < a.pairs && r < a.num_rows ? a.positions[static_cast<int64_t>(axis_row[i]) * a.num_rows + r] : 0;
  };
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int p = 32 * i + lane;
    my_turn[i] = p < a.pairs ? turn_of(a.freq[p]) : 0;
    axis_row[i] = p < a.pairs && a.axes ? min(max(a.axes[p], 0), a.num_axes - 1) : 0;
    pos[i] = position(i, row);
  }
  for (int c = 2 * a.pairs + lane; c < D; c += 32) {  // channels that are not turned
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint16_t* weight = k ? a.k_weight : a.q_weight;
      sm_coef[warp][k][0][c] = weight ? bf16(weight[c]) : 1.f;
      sm_coef[warp][k][1][c] = 0.f;
    }
  }
  int slot = 0;
#pragma unroll 1
  for (; row < a.num_rows; row += step) {
    __syncwarp();  // the last row's coefficients have been read
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int p = 32 * i + lane;
      if (p < a.pairs) {
        const float2 v = cos_sin(pos[i], my_turn[i]);
        const int c0 = kMode == kAdjacent ? 2 * p : p, c1 = kMode == kAdjacent ? 2 * p + 1 : p + a.pairs;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint16_t* weight = k ? a.k_weight : a.q_weight;
          const float w0 = weight ? bf16(weight[c0]) : 1.f, w1 = weight ? bf16(weight[c1]) : 1.f;
          sm_coef[warp][k][0][c0] = v.x * w0, sm_coef[warp][k][1][c0] = -v.y * w1;
          sm_coef[warp][k][0][c1] = v.x * w1, sm_coef[warp][k][1][c1] = v.y * w0;
        }
      }
      pos[i] = position(i, row + step);
    }
    __syncwarp();
    pair_t C[8], S[8];
#pragma unroll 1
    for (int turn = turn0; turn < turn1; ++turn) {
      const bool is_k = turn >= q_turns;
      if (turn == turn0 || turn == q_turns) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = 8 * (i < 2 ? pa : pb) + 4 * (i & 1);
          const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(&sm_coef[warp][is_k][0][c]);
          const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(&sm_coef[warp][is_k][1][c]);
          C[2 * i] = x.x, C[2 * i + 1] = x.y, S[2 * i] = y.x, S[2 * i + 1] = y.y;
        }
      }
      fetch();
      asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
      pair_t x[8], other[8];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 raw = ring[slot * 64 + 32 * i];
        x[4 * i] = unpack(raw.x), x[4 * i + 1] = unpack(raw.y);
        x[4 * i + 2] = unpack(raw.z), x[4 * i + 3] = unpack(raw.w);
      }
      slot = slot + 1 == kRing ? 0 : slot + 1;
      if constexpr (kMode == kHalvesAny) {
        float* sx = sm_x[warp][group];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float* at = sx + 9 * pa + 2 * i;
          at[0] = first(x[i]), at[1] = second(x[i]);
          other[i + 4] = 0;
        }
        const bool both = 4 * a.pairs > D;  // else none of the second pieces' channels is turned
        if (both) {
#pragma unroll
          for (int i = 4; i < 8; ++i) {
            float* at = sx + 9 * pb + 2 * (i - 4);
            at[0] = first(x[i]), at[1] = second(x[i]);
          }
        }
        __syncwarp();
        // channel e of piece p: its partner is `pairs` on, or back
        auto partner = [&](int p, int e) {
          const int c = 8 * p + e, on = e + a.pairs, back = e - a.pairs;
          return c < 2 * a.pairs ? sx[9 * p + (c < a.pairs ? on + (on >> 3) : back + (back >> 3))] : 0.f;
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) other[i] = pair(partner(pa, 2 * i), partner(pa, 2 * i + 1));
        if (both) {
#pragma unroll
          for (int i = 0; i < 4; ++i) other[i + 4] = pair(partner(pb, 2 * i), partner(pb, 2 * i + 1));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) other[i] = kMode == kHalves ? x[i ^ 4] : pair(second(x[i]), first(x[i]));
        if (2 * a.pairs < D) {
          // 0 times an infinity or NaN of another channel would reach one that is not turned
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (kMode == kHalves ? !turned : 4 * (i < 4 ? pa : pb) + (i & 3) >= a.pairs) other[i] = 0;
        }
      }
      const int head = (is_k ? turn - q_turns : turn) * kHeads + group;
      const bool live = head < (is_k ? a.Hkv : a.Hq);
      if (is_k ? a.k_weight : a.q_weight) {
        pair_t sum = mul(x[0], x[0]);
#pragma unroll
        for (int i = 1; i < 8; ++i) sum = fma(x[i], x[i], sum);
        float ss = first(sum) + second(sum);
#pragma unroll
        for (int off = kLanes / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
        const float v = ss * (1.f / D) + a.eps;
        float r = rsqrtf(v);
        if (live && !(v < INFINITY && (!kTiny || v >= kTinyEps))) {
          const bool large = !kTiny || !(v < 1.f);
          const float up = large ? 0x1p-96f : 0x1p96f;
          const uint32_t* raw = reinterpret_cast<const uint32_t*>(ring + (slot == 0 ? kRing - 1 : slot - 1) * 64);
          float y = 0.f;
#pragma unroll 1
          for (int i = 0; i < 8; ++i) {
            const pair_t two = unpack(raw[i < 4 ? i : 4 * 32 + i - 4]);
            y += first(two) * up * (first(two) * up) + second(two) * up * (second(two) * up);
          }
          const unsigned lanes = ((1u << (kLanes - 1) << 1) - 1u) << (group * kLanes);  // the head's
#pragma unroll
          for (int off = kLanes / 2; off > 0; off >>= 1) y += __shfl_xor_sync(lanes, y, off);
          r = rsqrtf(y * (1.f / D) + a.eps * up * up);
          if constexpr (kTiny) {
            // r times `up` may pass the largest number: the values take a share
            const float share = large ? 0x1p-32f : 0x1p96f;
            r *= large ? 0x1p-64f : 1.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = mul(x[i], pair(share, share)), other[i] = mul(other[i], pair(share, share));
          } else {
            r *= up;
          }
        }
        const pair_t rr = pair(r, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = mul(x[i], rr), other[i] = mul(other[i], rr);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = fma(other[i], S[i], mul(x[i], C[i]));
      if (live) {
        uint4* dst = reinterpret_cast<uint4*>((is_k ? a.k_out + row * a.k_out_stride : a.q_out + row * a.q_out_stride) + head * D);
        dst[pa] = make_uint4(pack(x[0]), pack(x[1]), pack(x[2]), pack(x[3]));
        dst[pb] = make_uint4(pack(x[4]), pack(x[5]), pack(x[6]), pack(x[7]));
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <int D>
cudaError_t launch(const RopeArgs& a, cudaStream_t stream) {
  constexpr int kHeads = 512 / D, kWarps = kRopeThreads / 32;
  const int turns = (a.Hq + kHeads - 1) / kHeads + (a.Hkv + kHeads - 1) / kHeads;
  // a row's heads go to several warps where there are too few rows to fill the SMs
  int dev = 0, sms = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  const int64_t most = sms * kRopeBlocks * kWarps;
  int parts = static_cast<int>(most / a.num_rows);
  parts = parts < 1 ? 1 : parts > turns ? turns : parts;
  const int per_part = (turns + parts - 1) / parts;
  parts = (turns + per_part - 1) / per_part;
  const int blocks = (a.num_rows - 1) / kWarps + 1, room = sms * kRopeBlocks / parts;
  const dim3 grid(blocks < room || room < 1 ? blocks : room, parts);
  auto go = [&](auto kernel) { return launch_dependent(kernel, grid, kRopeThreads, kWarps * kRing * 1024, stream, a, per_part); };
  auto go_mode = [&](auto tiny) {
    constexpr bool kTiny = decltype(tiny)::value;
    if (a.interleaved) return go(qk_rope_kernel<D, kAdjacent, kTiny>);
    if (a.pairs % 8 == 0) return go(qk_rope_kernel<D, kHalves, kTiny>);
    return go(qk_rope_kernel<D, kHalvesAny, kTiny>);
  };
  return a.eps < kTinyEps && (a.q_weight || a.k_weight) ? go_mode(std::true_type()) : go_mode(std::false_type());
}

}  // namespace

cudaError_t launch_qk_rope(const RopeArgs& a, cudaStream_t stream) {
  if (a.d == 64) return launch<64>(a, stream);
  if (a.d == 128) return launch<128>(a, stream);
  return launch<256>(a, stream);
}

}  // namespace bw
