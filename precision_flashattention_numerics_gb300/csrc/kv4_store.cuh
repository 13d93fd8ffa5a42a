// The 4-bit key/value cache: its format, storing rows in it (kv4_append_kernel) and reading
// them back (kv4_read_kernel).
//
// Format. A row of D channels is held as D / 2 bytes of codes (byte i: channel 2i in the low
// nibble, 2i + 1 in the high one) and D / 32 fp16 scales, one per group of 32 channels. With
// x = fp16_rn(K - shift) for keys (one shift per kv head and channel) and x = V for values,
// NaN counting as 0 and +-inf as +-65504:
//     s = fp16_rn(rn_8bits(max|x| / 7)),   c = clamp(rint_even(x / s), -7, 7) (0 where s = 0),
// stored as the nibble c + 8. s has 8 significant bits, so s * c (8 + 3 bits) is exactly an
// fp16 number and a reader that multiplies in fp16 rounds nothing.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "ptx.cuh"

namespace pasa {

constexpr int kKv4Group = 32;          // channels that share a scale
constexpr int kKv4StoreThreads = 256;

// Where a call's rows go: row i of sequence b (i < counts[b], or n) is cache row
// start[b] + i (or start + i); rows outside [0, cap) are skipped.
struct Kv4Window {
  const int* starts;   // device, or nullptr: `start` for every sequence
  const int* counts;   // device, or nullptr: n for every sequence
  int start, n, cap;
  // The cache row of row i of sequence b, or -1 where there is none.
  __device__ __forceinline__ long long row(int b, int i) const {
    const long long at = static_cast<long long>(starts ? starts[b] : start) + i;
    if (counts && i >= counts[b]) return -1;
    return at >= 0 && at < cap ? at : -1;
  }
};

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }

__device__ __forceinline__ float rcp_approx(float x) {   // within 2^-23
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// x rounded (ties to even) to 8 significant bits; x >= 0 and finite.
__device__ __forceinline__ float round_8bits(float x) {
  uint32_t u = __float_as_uint(x);
  u += 0x7FFFu + ((u >> 16) & 1u);
  return __uint_as_float(u & 0xFFFF0000u);
}

// The codes of 16 channels, one nibble each (bits 4i .. 4i + 3 of the first word: channel i), and the
// group's scale; x: 16 fp16 in 8 registers. Called by the 2 lanes of a group together (aligned
// pairs of lanes hold the 32 channels).
//
// Both quotients are only needed rounded, so products with reciprocals do. max|x| / 7 to 8 bits: a
// tie is a 9-bit number t with max|x| = 7 t; any other quotient of an 11-bit number is at least
// 2^-10 / 7 of t away from one. The product with 1 / 7, off by 2^-23, is first rounded to 16 bits:
// a true tie is then exact, and nothing else has moved onto or across one. x / s to an integer: where
// it is no tie (a multiple of 1/2), it is at least 2.4e-4 away from one: x has 11 significant bits,
// s 8, and both are multiples of a power of two no smaller than s * 2^-12. So x * (1 / s), off by
// at most 7 * 2^-22, is first rounded to a multiple of 2^-14 (by adding 768), and then to an integer
// (by adding 1.5 * 2^23 - 768), ties to even.
__device__ __forceinline__ uint2 kv4_codes(const uint32_t (&xin)[8], __half& scale) {
  uint32_t x[8];
  __half2 m2 = __float2half2_rn(0.0f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = xin[i];
    m2 = __hmax2_nan(m2, __habs2(bits_h2(x[i])));
  }
  m2 = __hmax2_nan(m2, __shfl_xor_sync(0xFFFFFFFFu, m2, 1));
  float a = __half2float(__hmax_nan(__low2half(m2), __high2half(m2)));
  // a group that is not finite, or so small that its scale has fewer than 8 bits and |x / s| may
  // pass 7 by more than rounding: the same in its 2 lanes
  const bool odd = !(a <= 65504.0f) || a < 7.0f * 0x1p-14f;
  const bool odds = __any_sync(0xFFFFFFFFu, odd);
  if (odds) {
    float b = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float2 f = __half22float2(bits_h2(x[i]));
      f.x = f.x == f.x ? fminf(fmaxf(f.x, -65504.0f), 65504.0f) : 0.0f;
      f.y = f.y == f.y ? fminf(fmaxf(f.y, -65504.0f), 65504.0f) : 0.0f;
      b = fmaxf(b, fmaxf(fabsf(f.x), fabsf(f.y)));
      x[i] = h2_bits(__float22half2_rn(f));
    }
    a = fmaxf(b, __shfl_xor_sync(0xFFFFFFFFu, b, 1));
  }
  const float sixteen_bits = __uint_as_float((__float_as_uint(a * (1.0f / 7.0f)) + 0x80u) & 0xFFFFFF00u);
  scale = __float2half_rn(round_8bits(sixteen_bits));
  if (odds) {
    const __half2 top = __hmul2(__half2half2(scale), __float2half2_rn(7.0f));
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = h2_bits(__hmax2(__hmin2(bits_h2(x[i]), top), __hneg2(top)));
  }
  const float s = __half2float(scale);
  const float r = s > 0.0f ? rcp_approx(s) : 0.0f;
  uint32_t w[2];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t b[4];   // low byte: two codes (1 .. 15 each)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(bits_h2(x[4 * half + i]));
      // 12582912 = 1.5 * 2^23: the integer code + 8 lands in the low bits of the float
      constexpr float kToInt = 12582912.0f + 8.0f - 768.0f;
      float lo, hi;
      ffma2(lo, hi, f.x, f.y, r, r, 768.0f, 768.0f);
      fadd2(lo, hi, lo, hi, kToInt, kToInt);
      b[i] = __float_as_uint(hi) * 16u + __float_as_uint(lo);
    }
    w[half] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
  }
  return make_uint2(w[0], w[1]);
}

// Rows of a thread, a block's rows apart; it takes the same channels of each, of K and V, of one
// (sequence, kv head) (blockIdx.y). Both kernels are HBM-bound: 4 D bytes of fp16 and 9 D / 8 of codes
// and scales per row, one way or the other. Storing, a thread takes 16 channels, so that two lanes
// have a group and its scale's arithmetic is shared by more (4 x 8 heads x 8192 rows, D = 128: 27.5 us,
// 0.93 of the copy rate; 36 us with 8 channels). Reading back, it takes 8, whose 16 bytes a warp
// stores without gaps (28.4 us; 41 us with 16, whose stores each fill half sectors).
constexpr int kKv4AppendRows = 2;
constexpr int kKv4ReadRows = 4;

__device__ __forceinline__ void load16(uint32_t (&x)[8], const __half* p) {
  const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p)), b = __ldcs(reinterpret_cast<const uint4*>(p) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// Store rows of k and v [B, H, n, D] in the cache.
template <int D>
__global__ void __launch_bounds__(kKv4StoreThreads) kv4_append_kernel(
    const __half* __restrict__ k, const __half* __restrict__ v, const __half* __restrict__ shift,
    uint8_t* __restrict__ k4, __half* __restrict__ kscale, uint8_t* __restrict__ v4, __half* __restrict__ vscale,
    int planes, int H, Kv4Window win) {
  griddep_launch_dependents();
  constexpr int kPer = D / 16;   // threads per row
  constexpr int kRows = kKv4StoreThreads / kPer, N = kKv4AppendRows;
  const int u = threadIdx.x % kPer;
  const int i0 = blockIdx.x * (N * kRows) + threadIdx.x / kPer;
  for (int plane = blockIdx.y; plane < planes; plane += gridDim.y) {
    const int b = plane / H;
    long long row[N];
    uint32_t xk[N][8] = {}, xv[N][8] = {};
    const __half* kp = k + (static_cast<long long>(plane) * win.n + i0) * D + u * 16;
    const __half* vp = v + (static_cast<long long>(plane) * win.n + i0) * D + u * 16;
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (i0 + j * kRows < win.n) {   // rows past counts too: waiting for the count first takes longer
        load16(xk[j], kp + j * kRows * D);
        load16(xv[j], vp + j * kRows * D);
      }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int i = i0 + j * kRows;
      row[j] = i < win.n ? win.row(b, i) : -1;
    }
    uint32_t sh[8] = {};   // x - 0 = x
    if (shift) load16(sh, shift + static_cast<long long>(plane) * D + u * 16);
#pragma unroll
    for (int j = 0; j < N; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) xk[j][i] = h2_bits(__hsub2_rn(bits_h2(xk[j][i]), bits_h2(sh[i])));
      __half sk, sv;
      const uint2 ck = kv4_codes(xk[j], sk), cv = kv4_codes(xv[j], sv);
      if (row[j] >= 0) {
        const long long at = static_cast<long long>(plane) * win.cap + row[j];
        *reinterpret_cast<uint2*>(k4 + at * (D / 2) + u * 8) = ck;
        *reinterpret_cast<uint2*>(v4 + at * (D / 2) + u * 8) = cv;
        if ((u & 1) == 0) {
          kscale[at * (D / kKv4Group) + u / 2] = sk;
          vscale[at * (D / kKv4Group) + u / 2] = sv;
        }
      }
    }
  }
}

// 8 codes (nibble i: channel i) times the scale, exactly, as 4 pairs (0, 4), (1, 5), (2, 6),
// (3, 7): a nibble masked into the mantissa of 1024 is 1024 + n, or 1024 + 16 n one place up.
__device__ __forceinline__ void kv4_expand(uint32_t w, __half2 s2, __half2 (&out)[4]) {
  const __half2 off0 = __float2half2_rn(-1032.0f), off1 = __float2half2_rn(-72.0f), sixteenth = __float2half2_rn(0.0625f);
  const uint32_t w8 = w >> 8;
  const uint32_t magic = 0x64006400u;
  out[0] = __hmul2(__hadd2(bits_h2((w & 0x000F000Fu) | magic), off0), s2);
  out[1] = __hmul2(__hfma2(bits_h2((w & 0x00F000F0u) | magic), sixteenth, off1), s2);
  out[2] = __hmul2(__hadd2(bits_h2((w8 & 0x000F000Fu) | magic), off0), s2);
  out[3] = __hmul2(__hfma2(bits_h2((w8 & 0x00F000F0u) | magic), sixteenth, off1), s2);
}

// 8 codes times the scale, exactly, in channel order.
__device__ __forceinline__ uint4 kv4_values8(uint32_t w, __half s) {
  __half2 p[4];
  kv4_expand(w, __half2half2(s), p);
  return make_uint4(h2_bits(__lows2half2(p[0], p[1])), h2_bits(__lows2half2(p[2], p[3])),
                    h2_bits(__highs2half2(p[0], p[1])), h2_bits(__highs2half2(p[2], p[3])));
}
__device__ __forceinline__ uint4 add8(uint4 x, uint4 y) {
  return make_uint4(h2_bits(__hadd2_rn(bits_h2(x.x), bits_h2(y.x))), h2_bits(__hadd2_rn(bits_h2(x.y), bits_h2(y.y))),
                    h2_bits(__hadd2_rn(bits_h2(x.z), bits_h2(y.z))), h2_bits(__hadd2_rn(bits_h2(x.w), bits_h2(y.w))));
}

// Read cache rows back as fp16: fp16_rn(s * c + shift) for keys, s * c for values, into
// k, v [B, H, n, D]; output rows without a cache row are left as they are.
template <int D>
__global__ void __launch_bounds__(kKv4StoreThreads) kv4_read_kernel(
    const uint8_t* __restrict__ k4, const __half* __restrict__ kscale, const uint8_t* __restrict__ v4,
    const __half* __restrict__ vscale, const __half* __restrict__ shift, __half* __restrict__ k,
    __half* __restrict__ v, int planes, int H, Kv4Window win) {
  constexpr int kPer = D / 8;   // threads per row
  constexpr int kRows = kKv4StoreThreads / kPer, N = kKv4ReadRows;
  const int u = threadIdx.x % kPer;
  const int i0 = blockIdx.x * (N * kRows) + threadIdx.x / kPer;
  for (int plane = blockIdx.y; plane < planes; plane += gridDim.y) {
    const int b = plane / H;
    long long row[N];
    uint32_t ck[N], cv[N];
    __half sk[N], sv[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int i = i0 + j * kRows;
      row[j] = i < win.n ? win.row(b, i) : -1;
      ck[j] = cv[j] = 0u;
      sk[j] = sv[j] = __ushort_as_half(0);
      if (row[j] >= 0) {
        const long long at = static_cast<long long>(plane) * win.cap + row[j];
        ck[j] = *reinterpret_cast<const uint32_t*>(k4 + at * (D / 2) + u * 4);
        cv[j] = *reinterpret_cast<const uint32_t*>(v4 + at * (D / 2) + u * 4);
        sk[j] = kscale[at * (D / kKv4Group) + u / 4];
        sv[j] = vscale[at * (D / kKv4Group) + u / 4];
      }
    }
    uint4 sh = make_uint4(0u, 0u, 0u, 0u);
    if (shift) sh = *reinterpret_cast<const uint4*>(shift + static_cast<long long>(plane) * D + u * 8);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (row[j] < 0) continue;
      const long long to = (static_cast<long long>(plane) * win.n + i0 + j * kRows) * D + u * 8;
      *reinterpret_cast<uint4*>(k + to) = add8(kv4_values8(ck[j], sk[j]), sh);
      *reinterpret_cast<uint4*>(v + to) = kv4_values8(cv[j], sv[j]);
    }
  }
}

}  // namespace pasa
