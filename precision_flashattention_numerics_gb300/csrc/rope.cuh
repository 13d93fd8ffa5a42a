// Rotary positions: the first R of a row's D channels are turned in pairs by angles that grow with
// the token's position.
//
// A pair (x, y) of a token at position p becomes (x c - y s, x s + y c), c = mscale cos a, s = mscale
// sin a, a = p * inv_freq[i]; pairs are (i, i + R / 2) (the half layout) or (2i, 2i + 1) (interleaved).
// Backwards (the transpose, which is also the gradient) with -s.
//
// The angle. In fp32 the product p * inv_freq is off by half a unit of its last place, 0.03 radians
// at p = 10^6; in fp64 it takes the few fp64 units of an SM as long as the whole kernel. Only
// the fraction of a turn counts, so inv_freq / 2 pi is held as a 64-bit fraction of a turn and p times
// it is one 64-bit integer product, whose overflow drops whole turns. Its upper 32 bits are the
// fraction in units of 2^-32, and sinpi and cospi of them in fp32 are off by 2^-23 or so at
// any position. (inv_freq / 2 pi itself is made in integers: rounded to fp64, the farthest
// positions are off by 2^-22.8 radians at 1 radian a position, and by 2^-12 at 1000.)
//
// HBM-bound: every channel is read once and written once, with 16-byte accesses. A CTA takes a few tokens: its threads make the
// cos and sin of their angles in shared memory, then a thread takes two vectors of 8 channels, which hold 8 whole
// pairs in either layout, of one token and every `slots`-th head, with the angles in registers and the rows of two
// heads on their way at a time, which leaves registers for 4 CTAs on an SM. The table of fractions is made once per CTA.
// Measured, 32768 tokens x 32 heads x 128 in fp16: 96 us for 537 MB, 0.83 of the copy rate (angles made by every thread for
// 4 heads: 152 us; 4 heads at a time and 2 CTAs: 150; 1 head and 8 CTAs, which spills: 210).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"

namespace pasa {

constexpr int kRopeThreads = 256;
constexpr int kRopeHeads = 2;   // of a thread, on their way at a time
constexpr int kRopeMaxD = 256;

// One tensor [B, H, S, D], channels contiguous; strides in elements.
struct RopeTensor {
  const void* in;
  void* out;
  long long in_b, in_h, in_s, out_b, out_h, out_s;
};

struct RopeParams {
  RopeTensor t[2];          // q and k
  int Hq, heads;            // heads of q, and of both
  const double* inv_freq;   // [R / 2] radians per position
  const int* positions;     // [B, S], or nullptr:
  const int* starts;        // [B], or nullptr: token s of sequence b is at starts[b] (or start) + s
  int start;
  int S, D, R;
  unsigned tokens, slots, groups;   // B * S; head slots of a token; channel groups of a row
  unsigned token0;                  // rope_pairs_kernel: the launch's tokens are token0 .. tokens - 1
  unsigned cta_tokens;              // of a CTA: kRopeThreads / (groups * slots), or 1
  float mscale, sign;
};

// The fraction of a turn per position as a 64-bit fixed-point number, cut off, and cos and sin of p times it. The number's 53-bit
// mantissa times 1 / 2 pi to 128 bits, in integers, and shifted by its exponent: no rounding, and no fp64 unit.
__device__ __forceinline__ unsigned long long rope_turns(double inv_freq) {
  using u64 = unsigned long long;
  constexpr u64 kHigh = 0xA2F9836E4E441529, kLow = 0xFC2757D1F534DDC0;   // 2^130 / 2 pi
  const u64 bits = static_cast<u64>(__double_as_longlong(inv_freq));
  const int shift = 66 + 1075 - static_cast<int>(bits >> 52 & 0x7FF);
  if (shift < 0 || shift >= 192) return 0;   // below 2^-64 of a turn; from 2^119 radians on, infinite or NaN
  const u64 m = (bits & 0xFFFFFFFFFFFFF) | 0x10000000000000;
  const u64 p0 = m * kLow, p1 = m * kHigh + __umul64hi(m, kLow), p2 = __umul64hi(m, kHigh) + (p1 < m * kHigh ? 1 : 0);
  const int word = shift >> 6, r = shift & 63;
  const u64 low = word == 0 ? p0 : word == 1 ? p1 : p2, high = word == 0 ? p1 : word == 1 ? p2 : 0;
  const u64 turns = low >> r | (high << 1) << (63 - r);
  return bits >> 63 ? 0 - turns : turns;
}
__device__ __forceinline__ void rope_angle(unsigned long long turns, long long p, float mscale, float sign, float& c, float& s) {
  const unsigned long long a = turns * static_cast<unsigned long long>(p);
  // half turns in [-1, 1)
  const float x = static_cast<float>(static_cast<int>(a >> 32)) * 0x1p-31f;
  sincospif(x, &s, &c);
  c *= mscale;
  s *= mscale * sign;
}

// A start and its tokens may pass 32 bits.
__device__ __forceinline__ long long rope_position(const RopeParams& p, unsigned token, unsigned b, unsigned s) {
  if (p.positions) return p.positions[token];
  return static_cast<long long>(p.starts ? p.starts[b] : p.start) + s;
}

// 8 channels as they are in memory, as fp32, and back with one rounding each.
template <typename T>
struct RopeRaw {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) v[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
};
__device__ __forceinline__ void rope_values(float (&x)[8], const RopeRaw<__half>& r) {
  const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = f.x, x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void rope_values(float (&x)[8], const RopeRaw<__nv_bfloat16>& r) {
  const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
}
__device__ __forceinline__ void rope_values(float (&x)[8], const RopeRaw<float>& r) {
  const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
}
__device__ __forceinline__ void rope_store8(__half* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]), pack_half2(x[4], x[5]), pack_half2(x[6], x[7]));
}
__device__ __forceinline__ void rope_store8(__nv_bfloat16* p, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void rope_store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ float rope_get(__half x) { return __half2float(x); }
__device__ __forceinline__ float rope_get(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float rope_get(float x) { return x; }
__device__ __forceinline__ void rope_put(__half* p, float x) { *p = __float2half_rn(x); }
__device__ __forceinline__ void rope_put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void rope_put(float* p, float x) { *p = x; }

// R a multiple of 16, D of 8, rows on 16-byte boundaries. Group g < R / 16 is 8 pairs; those behind them are 16
// channels that are only copied (none of them where every tensor is turned in place).
template <typename TIn, typename TOut, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ unsigned long long turns[kRopeMaxD / 2];
  __shared__ float2 angles[kRopeThreads * 8];   // [token of the CTA][pair]; a CTA's groups hold 8 pairs each
  const unsigned g = threadIdx.x % p.groups, rest = threadIdx.x / p.groups;
  const unsigned slot = rest % p.slots, t0 = rest / p.slots;
  const unsigned first = blockIdx.x * p.cta_tokens, token = first + t0;
  const bool live = t0 < p.cta_tokens && token < p.tokens;
  const unsigned b = token / p.S, s = token - b * p.S;
  const unsigned pairs = p.R / 2;
  const bool turn = g * 8 < pairs;
  // channels of the two vectors
  const int c0 = turn && !INTERLEAVED ? 8 * g : 16 * g;
  const int c1 = turn && !INTERLEAVED ? pairs + 8 * g : 16 * g + 8;
  const bool two = c1 < p.D;
  auto row = [&](int head, bool out) -> long long {   // of an existing head: elements from its tensor's start
    const RopeTensor& t = p.t[head >= p.Hq ? 1 : 0];
    const int h = head >= p.Hq ? head - p.Hq : head;
    return out ? b * t.out_b + h * t.out_h + s * t.out_s : b * t.in_b + h * t.in_h + s * t.in_s;
  };
  RopeRaw<TIn> x[kRopeHeads][2];
  auto load = [&](int head0) {
#pragma unroll
    for (int j = 0; j < kRopeHeads; ++j) {
      const int head = head0 + j * p.slots;
      if (!live || head >= p.heads) continue;
      const TIn* in = static_cast<const TIn*>(p.t[head >= p.Hq ? 1 : 0].in) + row(head, false);
      x[j][0].load(in + c0);
      if (two) x[j][1].load(in + c1);
    }
  };
  load(slot);   // on their way while the angles are made
  if (threadIdx.x < pairs) turns[threadIdx.x] = rope_turns(p.inv_freq[threadIdx.x]);
  __syncthreads();
  for (unsigned i = threadIdx.x; i < p.cta_tokens * pairs; i += kRopeThreads) {
    const unsigned tok = first + i / pairs, pair = i % pairs;
    if (tok >= p.tokens) break;
    const unsigned tb = tok / p.S;
    float2 cs;
    rope_angle(turns[pair], rope_position(p, tok, tb, tok - tb * p.S), p.mscale, p.sign, cs.x, cs.y);
    angles[i] = cs;
  }
  __syncthreads();
  if (!live) return;
  float2 cs[8];
  if (turn) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float4 a = *reinterpret_cast<const float4*>(&angles[t0 * pairs + 8 * g + i]);
      cs[i] = make_float2(a.x, a.y), cs[i + 1] = make_float2(a.z, a.w);
    }
  }
  for (int head0 = slot; head0 < p.heads; head0 += kRopeHeads * p.slots) {
    if (head0 != static_cast<int>(slot)) load(head0);
#pragma unroll
    for (int j = 0; j < kRopeHeads; ++j) {
      const int head = head0 + j * p.slots;
      if (head >= p.heads) continue;
      float y[2][8] = {};
      rope_values(y[0], x[j][0]);
      if (two) rope_values(y[1], x[j][1]);
      if (turn) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float& u = INTERLEAVED ? y[i / 4][2 * (i % 4)] : y[0][i];
          float& v = INTERLEAVED ? y[i / 4][2 * (i % 4) + 1] : y[1][i];
          const float z = u * cs[i].x - v * cs[i].y;
          v = u * cs[i].y + v * cs[i].x;
          u = z;
        }
      }
      TOut* out = static_cast<TOut*>(p.t[head >= p.Hq ? 1 : 0].out) + row(head, true);
      rope_store8(out + c0, y[0]);
      if (two) rope_store8(out + c1, y[1]);
    }
  }
}

// Any even R and any strides: a thread takes one pair, or one channel behind the R, of one token and head. Threads of a launch are
// counted in 32 bits; larger calls are launched in parts of whole tokens.
template <typename TIn, typename TOut, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_pairs_kernel(const __grid_constant__ RopeParams p) {
  __shared__ unsigned long long turns[kRopeMaxD / 2];
  if (threadIdx.x < p.R / 2) turns[threadIdx.x] = rope_turns(p.inv_freq[threadIdx.x]);
  __syncthreads();
  const unsigned id = blockIdx.x * kRopeThreads + threadIdx.x;
  const unsigned row = id / p.groups, g = id - row * p.groups;
  const unsigned t0 = row / p.slots, head = row - t0 * p.slots, token = p.token0 + t0;
  if (token >= p.tokens) return;
  const unsigned b = token / p.S, s = token - b * p.S;
  const RopeTensor& t = p.t[static_cast<int>(head) >= p.Hq ? 1 : 0];
  const int h = static_cast<int>(head) >= p.Hq ? head - p.Hq : head;
  const TIn* in = static_cast<const TIn*>(t.in) + b * t.in_b + h * t.in_h + s * t.in_s;
  TOut* out = static_cast<TOut*>(t.out) + b * t.out_b + h * t.out_h + s * t.out_s;
  const int pairs = p.R / 2;
  if (static_cast<int>(g) >= pairs) {
    const int c = p.R + g - pairs;
    rope_put(out + c, rope_get(in[c]));
    return;
  }
  const int c0 = INTERLEAVED ? 2 * g : g, c1 = INTERLEAVED ? 2 * g + 1 : g + pairs;
  const float u = rope_get(in[c0]), v = rope_get(in[c1]);
  float c, sn;
  rope_angle(turns[g], rope_position(p, token, b, s), p.mscale, p.sign, c, sn);
  rope_put(out + c0, u * c - v * sn);
  rope_put(out + c1, u * sn + v * c);
}

}  // namespace pasa
