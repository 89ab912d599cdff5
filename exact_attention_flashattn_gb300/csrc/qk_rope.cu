// Norm and rotation of queries and keys in one pass, rows of a projection in, q and k for attention out:
//   n_c = x_c w_c / sqrt(mean x^2 + eps)            (a head's d channels; without a weight n = x)
//   (a, b) -> (a cos t - b sin t, a sin t + b cos t)  for each pair of channels, t = position * frequency,
// pairs (c, c + pairs) or, interleaved, (2 c, 2 c + 1); the position comes from the pair's axis (time, height,
// width). Channels behind the pairs are normalised only. 32 bits in between, rounded to bf16 once.
//
// What bounds it: every value is read and written once, 4 bytes each. A warp takes whole rows, some heads of
// one at a time: d / 16 lanes a head, each with two pieces of 8 channels that hold both halves of its pairs,
// so rotating needs no exchange.
#include "kernels.h"
#include "ptx.cuh"

namespace bw {

namespace {

constexpr int kSms = 152;
constexpr int kRopeThreads = 128;

enum RopeMode { kHalves, kAdjacent, kHalvesAny };  // kHalvesAny: pairs no multiple of 8

// A rotation's angle in turns is position * frequency / 2 pi modulo 1: with the frequency as a fraction of 2^64
// the product of integers wraps to just that, however far the position. The frequency's own rounding, 2^-53 of
// it, is off by less than the angle's rounding to 32 bits up to positions of 2^28 or so.
__device__ __forceinline__ uint64_t turn_of(float freq) {
  const double t = static_cast<double>(freq) * 0.15915494309189535;  // 1 / 2 pi
  return __double2ull_rd((t - floor(t)) * 0x1p64);
}
__device__ __forceinline__ float2 cos_sin(int position, uint64_t turn) {
  const uint64_t x = static_cast<uint64_t>(static_cast<int64_t>(position)) * turn;
  float s, c;
  sincospif(static_cast<float>(static_cast<int32_t>(x >> 32)) * 0x1p-31f, &s, &c);
  return make_float2(c, s);
}

__device__ __forceinline__ void unpack(const uint4& u, float* x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(w[e] << 16);
    x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack(const float* x) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

template <int D, int kMode>
__global__ void __launch_bounds__(kRopeThreads) qk_rope_kernel(const RopeArgs a, int parts, int per_part) {
  constexpr int kLanes = D / 16, kHeads = 32 / kLanes;  // lanes a head, heads a turn
  constexpr int kPairs = D / 2, kMine = kPairs / 32;    // table entries, a lane's
  constexpr int kWarps = kRopeThreads / 32;
  __shared__ float2 sm_table[kWarps][kPairs];
  __shared__ float sm_x[kMode == kHalvesAny ? kWarps : 1][kMode == kHalvesAny ? kHeads : 1][kMode == kHalvesAny ? D : 1];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = lane % kLanes, group = lane / kLanes;
  float2* table = sm_table[warp];
  // what a lane keeps over its rows: the turns of its table entries, the weights of its channels
  uint64_t turn[kMine];
  int axis[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int pair = 32 * i + lane;
    turn[i] = pair < a.pairs ? turn_of(a.freq[pair]) : 0;
    axis[i] = pair < a.pairs && a.axes ? min(max(a.axes[pair], 0), a.num_axes - 1) : 0;
  }
  // the two pieces: both halves of 8 pairs, or neighbours among the channels that are not turned
  const int p8 = a.pairs / 8;
  const int pa = kMode == kHalves ? (t < p8 ? t : 2 * t) : t;
  const int pb = kMode == kHalves ? (t < p8 ? t + p8 : 2 * t + 1) : t + kLanes;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  uint4 wq[2] = {zero, zero}, wk[2] = {zero, zero};
  if (a.q_weight) {
    wq[0] = reinterpret_cast<const uint4*>(a.q_weight)[pa];
    wq[1] = reinterpret_cast<const uint4*>(a.q_weight)[pb];
  }
  if (a.k_weight) {
    wk[0] = reinterpret_cast<const uint4*>(a.k_weight)[pa];
    wk[1] = reinterpret_cast<const uint4*>(a.k_weight)[pb];
  }
  const int heads = a.Hq + a.Hkv;
  const int64_t items = static_cast<int64_t>(a.num_rows) * parts;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + warp; item < items; item += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int64_t row = item / parts;
    const int h0 = static_cast<int>(item - row * parts) * per_part, h1 = min(h0 + per_part, heads);
    __syncwarp();  // the last row's table has been read
#pragma unroll
    for (int i = 0; i < kMine; ++i)
      // a pair that is not turned: (1, 0)
      table[32 * i + lane] = 32 * i + lane < a.pairs
                                 ? cos_sin(a.positions[static_cast<int64_t>(axis[i]) * a.num_rows + row], turn[i])
                                 : make_float2(1.f, 0.f);
    __syncwarp();
    float2 cs[8];
    if constexpr (kMode != kHalvesAny) {
#pragma unroll
      for (int e = 0; e < 8; ++e) cs[e] = table[kMode == kHalves ? 8 * t + e : 4 * (e < 4 ? pa : pb) + (e & 3)];
    }
#pragma unroll 2
    for (int h = h0; h < h1; h += kHeads) {
      const int head = h + group;
      const bool is = head < h1, is_k = head >= a.Hq;
      const uint16_t* src = is_k ? a.k + row * a.k_stride + (head - a.Hq) * D : a.q + row * a.q_stride + head * D;
      uint4 u[2] = {zero, zero};
      if (is) {
        u[0] = reinterpret_cast<const uint4*>(src)[pa];
        u[1] = reinterpret_cast<const uint4*>(src)[pb];
      }
      float x[16];
      unpack(u[0], x);
      unpack(u[1], x + 8);
      const bool norm = is_k ? a.k_weight != nullptr : a.q_weight != nullptr;
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
      for (int off = kLanes / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
      if (norm) {
        const float r = rsqrtf(ss * (1.f / D) + a.eps);
        float w[16];
        unpack(is_k ? wk[0] : wq[0], w);
        unpack(is_k ? wk[1] : wq[1], w + 8);
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = x[e] * r * w[e];
      }
      float y[16];
      if constexpr (kMode == kHalves) {
        const bool turned = t < p8;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          y[e] = turned ? x[e] * cs[e].x - x[e + 8] * cs[e].y : x[e];
          y[e + 8] = turned ? x[e] * cs[e].y + x[e + 8] * cs[e].x : x[e + 8];
        }
      } else if constexpr (kMode == kAdjacent) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const bool turned = 4 * (e < 4 ? pa : pb) + (e & 3) < a.pairs;
          y[2 * e] = turned ? x[2 * e] * cs[e].x - x[2 * e + 1] * cs[e].y : x[2 * e];
          y[2 * e + 1] = turned ? x[2 * e] * cs[e].y + x[2 * e + 1] * cs[e].x : x[2 * e + 1];
        }
      } else {
        float* sx = sm_x[warp][group];
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 16; ++e) sx[8 * (e < 8 ? pa : pb) + (e & 7)] = x[e];
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int c = 8 * (e < 8 ? pa : pb) + (e & 7);
          y[e] = x[e];
          if (c < a.pairs) {
            y[e] = x[e] * table[c].x - sx[c + a.pairs] * table[c].y;
          } else if (c < 2 * a.pairs) {
            y[e] = sx[c - a.pairs] * table[c - a.pairs].y + x[e] * table[c - a.pairs].x;
          }
        }
      }
      if (is) {
        uint16_t* dst = is_k ? a.k_out + row * a.k_out_stride + (head - a.Hq) * D : a.q_out + row * a.q_out_stride + head * D;
        reinterpret_cast<uint4*>(dst)[pa] = pack(y);
        reinterpret_cast<uint4*>(dst)[pb] = pack(y + 8);
      }
    }
  }
}

template <int D>
cudaError_t launch(const RopeArgs& a, cudaStream_t stream) {
  constexpr int kHeads = 512 / D, kWarps = kRopeThreads / 32;
  const int turns = (a.Hq + a.Hkv + kHeads - 1) / kHeads;
  // a row's heads go to several warps where there are too few rows to fill the SMs
  const int64_t want = static_cast<int64_t>(kSms) * 32;
  int parts = static_cast<int>(want / a.num_rows < 1 ? 1 : want / a.num_rows);
  if (parts > turns) parts = turns;
  const int per_turns = (turns + parts - 1) / parts;
  parts = (turns + per_turns - 1) / per_turns;
  const int64_t blocks = (static_cast<int64_t>(a.num_rows) * parts + kWarps - 1) / kWarps;
  const dim3 grid(static_cast<unsigned>(blocks < kSms * 16 ? blocks : kSms * 16));
  auto go = [&](auto kernel) { return launch_dependent(kernel, grid, kRopeThreads, 0, stream, a, parts, per_turns * kHeads); };
  if (a.interleaved) return go(qk_rope_kernel<D, kAdjacent>);
  if (a.pairs % 8 == 0) return go(qk_rope_kernel<D, kHalves>);
  return go(qk_rope_kernel<D, kHalvesAny>);
}

}  // namespace

cudaError_t launch_qk_rope(const RopeArgs& a, cudaStream_t stream) {
  if (a.d == 64) return launch<64>(a, stream);
  if (a.d == 128) return launch<128>(a, stream);
  return launch<256>(a, stream);
}

}  // namespace bw
