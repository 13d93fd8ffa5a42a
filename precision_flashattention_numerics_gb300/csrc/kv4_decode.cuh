// Decode attention on the 4-bit cache of kv4_store.cuh: a few query rows per head against
// cached keys and values, O = softmax(scale * q K'^T) V, and the attention weight each cached
// row gets. One shift per kv head and channel is the same for every key of a row, so
// q . shift cancels in the softmax and only enters the log-sum-exp.
//
// kv4_decode_kernel. HBM-bound: 9 D / 8 bytes per cached row of K and V against 4 rows D
// flops. A warp takes 32 keys at a time from global memory straight into registers and
// multiplies with mma.sync m16n8k16 (fp16 in, fp32 out):
//   S^T[key][row] = K' Q^T:  A = K' (16 keys x 16 channels), B = Q^T (16 channels x 8 rows);
//   O^T[channel][row] += V^T P^T:  A = V^T (16 channels x 16 keys), B = P^T (16 keys x 8 rows).
// tcgen05 takes its operands from shared or tensor memory, so the expanded codes (4 times the
// bytes that HBM delivers) would cross shared memory twice; the register operands of mma.sync
// need neither trip, and with 8 or 16 rows the tensor work is small. Channels and
// keys are numbered inside an MMA so that a thread's operands are the consecutive bytes it
// loads: lane (g, t) = (lane / 4, lane % 4) loads channels t * D/4 .. of keys g, g + 8, .. for
// S and channels g * D/8 .. of keys 2t, 2t + 1, .. for O. S^T comes out with keys along the
// lanes' g and P^T is needed with keys along t: one movmatrix per 8 x 8 block.
// Every code times its scale is exact in fp16 (the scale has 8 significant bits), so K' and V
// enter the MMAs as the cache's values themselves; P is rounded to fp16 (relative 2^-11, as in
// the other decode kernels); scores, maxima, sums and O stay fp32.
//
// Work split. With `stream_k` the 32-key units of all (sequence, kv head, row tile) segments
// are numbered in order and CTA c takes the c-th of gridDim.x equal ranges, so uneven lengths
// keep all SMs equally busy. A segment inside one CTA is finished there; otherwise its CTAs
// leave (O, max, sum) partials and kv4_merge_kernel joins them. Without it, CTA s takes segment
// s whole: one launch, no workspace.
#pragma once

#include <cmath>
#include <cstdint>
#include <cuda_fp16.h>

#include "kv4_store.cuh"
#include "ptx.cuh"

namespace pasa {

constexpr int kKv4Warps = 8;
constexpr int kKv4Unit = 32;    // keys a warp takes at a time

struct Kv4Params {
  const __half* q;
  const uint8_t *k4, *v4;
  const __half *kscale, *vscale, *shift;   // shift: [B, Hkv, D] or nullptr
  const int* lengths;                      // [B] or nullptr: Sk rows in every sequence
  __half* o;
  float* lse;        // or nullptr
  float* weights;    // [B, Hkv, cap] or nullptr
  float* part_o;     // [gridDim.x + segments][tile rows][D]
  float2* part_ml;   // [gridDim.x + segments][tile rows]: max (log2 units), sum
  float* lse2;       // [segments][tile rows]: log2-sum-exp2 of the shifted scores, for the weights pass
  int B, Hkv, g, Sq, rows, row_tiles;      // rows = g * Sq query rows of a kv head
  int Sk, cap, causal;
  int len_add;       // added to lengths[] (a step call appends that many rows first)
  int ctas;          // gridDim.x of the decode kernel
  float scale, scale_log2;

  __device__ __forceinline__ int length(int b) const {
    if (!lengths) return Sk;
    const long long n = static_cast<long long>(lengths[b]) + len_add;
    return n < 0 ? 0 : n > Sk ? Sk : static_cast<int>(n);
  }
  // Keys row r of a kv head sees in a sequence of len keys (bottom-right aligned mask).
  __device__ __forceinline__ int limit(int r, int len) const {
    if (!causal) return len;
    const int n = r % Sq + len - Sq + 1;
    return n < 0 ? 0 : n;
  }
};

__device__ __forceinline__ int kv4_units(int len) { return (len + kKv4Unit - 1) / kKv4Unit; }

// Units of all sequences (per kv head and row tile), summed by a whole warp.
__device__ __forceinline__ long long kv4_sum_units(const Kv4Params& p, int b_end) {
  if (!p.lengths) return static_cast<long long>(b_end) * kv4_units(p.Sk);
  long long n = 0;
  for (int b = threadIdx.x & 31; b < b_end; b += 32) n += kv4_units(p.length(b));
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, d);
  return n;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// Codes and scales stream past once: no L1 line is kept for them.
template <int N>
__device__ __forceinline__ void ldg_words(uint32_t (&d)[N], const void* p) {
  if constexpr (N == 4)
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3]) : "l"(p));
  else if constexpr (N == 2)
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(d[0]), "=r"(d[1]) : "l"(p));
  else
    asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(d[0]) : "l"(p));
}
__device__ __forceinline__ uint32_t ldg_half(const __half* p) {
  uint16_t d;
  asm volatile("ld.global.u16 %0, [%1];" : "=h"(d) : "l"(p));
  return d;
}

// A warp's codes and scales of 32 keys of one head. Keys past the sequence's last are not
// read: their scale is 0, and so are their values, whatever the memory holds.
template <int D>
struct Kv4Keys {
  static constexpr int W = D / 32;   // 32-bit words of a lane's channels
  uint32_t k[4][W], ks[4];           // keys g + 8 i
  __device__ __forceinline__ void load(const uint8_t* k4, const __half* kscale, long long key0, int left, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const uint8_t* kp = k4 + (key0 + g) * (D / 2) + t * (D / 8);
    const __half* sp = kscale + (key0 + g) * (D / 32) + t * (D / 32) / 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (g + 8 * i < left) {
        ldg_words(k[i], kp + i * 8 * (D / 2));
        ks[i] = ldg_half(sp + i * 8 * (D / 32));
      } else {
#pragma unroll
        for (int w = 0; w < W; ++w) k[i][w] = 0;
        ks[i] = 0;
      }
    }
  }
};

template <int D>
struct Kv4Values {
  static constexpr int W = D / 64;
  uint32_t v[8][W], vs[8];           // keys 16 (j / 4) + 2t + j % 2 + 8 (j / 2 % 2)
  __device__ __forceinline__ void load(const uint8_t* v4, const __half* vscale, long long key0, int left, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const uint8_t* vp = v4 + (key0 + 2 * t) * (D / 2) + g * (D / 16);
    const __half* sp = vscale + (key0 + 2 * t) * (D / 32) + g * (D / 32) / 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int key = 16 * (j / 4) + (j & 1) + 8 * ((j >> 1) & 1);
      if (2 * t + key < left) {
        ldg_words(v[j], vp + key * (D / 2));
        vs[j] = ldg_half(sp + key * (D / 32));
      } else {
#pragma unroll
        for (int w = 0; w < W; ++w) v[j][w] = 0;
        vs[j] = 0;
      }
    }
  }
};

// The B operands of S for 8 query rows: lane (g, t) holds channels t * D/4 .. of row g in the
// order the expanded codes have.
template <int D>
__device__ __forceinline__ void kv4_query(uint32_t (&q)[D / 16][2], const __half* rows, int n, int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int w = 0; w < D / 32; ++w) {
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (g < n) x = *reinterpret_cast<const uint4*>(rows + g * D + t * (D / 4) + 8 * w);
    q[2 * w][0] = __byte_perm(x.x, x.z, 0x5410);       // channels 0, 4
    q[2 * w][1] = __byte_perm(x.x, x.z, 0x7632);       // 1, 5
    q[2 * w + 1][0] = __byte_perm(x.y, x.w, 0x5410);   // 2, 6
    q[2 * w + 1][1] = __byte_perm(x.y, x.w, 0x7632);   // 3, 7
  }
}

// S^T of 16 keys (half s of the unit) and NT * 8 rows.
template <int D, int NT>
__device__ __forceinline__ void kv4_scores(float (&acc)[NT][4], const Kv4Keys<D>& kk, int s,
                                           const uint32_t (&q)[NT][D / 16][2]) {
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[nt][e] = 0.0f;
  const __half2 sa = bits_h2(__byte_perm(kk.ks[2 * s], 0, 0x1010));
  const __half2 sb = bits_h2(__byte_perm(kk.ks[2 * s + 1], 0, 0x1010));
#pragma unroll
  for (int w = 0; w < D / 32; ++w) {
    __half2 a[4], b[4];
    kv4_expand(kk.k[2 * s][w], sa, a);
    kv4_expand(kk.k[2 * s + 1][w], sb, b);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      mma_f16(acc[nt], h2_bits(a[0]), h2_bits(b[0]), h2_bits(a[1]), h2_bits(b[1]), q[nt][2 * w][0], q[nt][2 * w][1]);
      mma_f16(acc[nt], h2_bits(a[2]), h2_bits(b[2]), h2_bits(a[3]), h2_bits(b[3]), q[nt][2 * w + 1][0],
              q[nt][2 * w + 1][1]);
    }
  }
}

// Finish a row: O and LSE from sum, max and the unnormalised O held in shared or global memory.
__device__ __forceinline__ float kv4_lse(float m, float l, float offset) {
  return l == 0.0f ? -INFINITY : 0.69314718055994531f * (m + log2f(l)) + offset;
}

template <int D, int NT>
struct Kv4Smem {
  float o[kKv4Warps][NT * 8][D + 4];
  float m[kKv4Warps][NT * 8], l[kKv4Warps][NT * 8];
  float factor[kKv4Warps][NT * 8];
  float row_m[NT * 8], row_l[NT * 8], offset[NT * 8];
};

// scale * q . shift of a row (natural-log units), by a whole warp.
template <int D>
__device__ __forceinline__ float kv4_offset(const Kv4Params& p, long long bh, int r, int lane) {
  if (!p.shift) return 0.0f;
  const __half* q = p.q + (bh * p.rows + r) * D;
  const __half* m = p.shift + bh * D;
  float s = 0.0f;
#pragma unroll
  for (int c = 0; c < D; c += 32) s = fmaf(__half2float(q[c + lane]), __half2float(m[c + lane]), s);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
  return s * p.scale;
}

template <int D, int NT, bool STREAM_K>
__global__ void __launch_bounds__(kKv4Warps * 32, NT == 1 ? 2 : 1) kv4_decode_kernel(Kv4Params p) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Kv4Smem<D, NT>& sm = *reinterpret_cast<Kv4Smem<D, NT>*>(smem_raw);
  constexpr int kRows = NT * 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  griddep_launch_dependents();
  griddep_wait();   // rows that the call's append kernel stores

  // this CTA's segments: (b, h, row tile) in order, and the units [u0, u1) of the first
  long long u_begin = 0, u_end = 0;
  int b = 0, u0 = 0, n_units = 0, len = 0;
  long long in_b = 0;   // segment inside sequence b: h * row_tiles + row tile
  const long long per_b = static_cast<long long>(p.Hkv) * p.row_tiles;
  if (STREAM_K) {
    const long long total = kv4_sum_units(p, p.B) * per_b;
    const long long ctas = total < gridDim.x ? total : gridDim.x;
    if (blockIdx.x >= ctas) return;
    u_begin = static_cast<long long>(blockIdx.x) * total / ctas;
    u_end = (static_cast<long long>(blockIdx.x) + 1) * total / ctas;
    long long before = 0;
    for (;; ++b) {
      len = p.length(b);
      n_units = kv4_units(len);
      if (before + n_units * per_b > u_begin) break;
      before += n_units * per_b;
    }
    in_b = (u_begin - before) / n_units;
    u0 = static_cast<int>((u_begin - before) % n_units);
  } else {
    b = static_cast<int>(blockIdx.x / per_b);
    in_b = blockIdx.x % per_b;
    len = p.length(b);
    n_units = kv4_units(len);
    u_end = n_units;
  }

  while (true) {
    const long long bh = static_cast<long long>(b) * p.Hkv + in_b / p.row_tiles;
    const int row0 = static_cast<int>(in_b % p.row_tiles) * kRows;
    const int n_rows = min(kRows, p.rows - row0);
    const int u1 = static_cast<int>(min(static_cast<long long>(n_units), u0 + (u_end - u_begin)));

    // ---- the warp's share of units u0 .. u1 ----
    uint32_t q[NT][D / 16][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      kv4_query<D>(q[nt], p.q + (bh * p.rows + row0 + nt * 8) * D, n_rows - nt * 8, lane);
    float o[NT][D / 16][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.0f;
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.0f;
    }
    const uint8_t* k4 = p.k4 + bh * p.cap * (D / 2);
    const uint8_t* v4 = p.v4 + bh * p.cap * (D / 2);
    const __half* kscale = p.kscale + bh * p.cap * (D / 32);
    const __half* vscale = p.vscale + bh * p.cap * (D / 32);
    const int all_see = p.causal ? max(0, len - p.Sq + 1) : len;   // keys that every row sees

    Kv4Keys<D> kk;
    Kv4Values<D> vv;
    int u = u0 + warp;
    if (u < u1) {
      kk.load(k4, kscale, static_cast<long long>(u) * kKv4Unit, len - u * kKv4Unit, lane);
      vv.load(v4, vscale, static_cast<long long>(u) * kKv4Unit, len - u * kKv4Unit, lane);
    }
    for (; u < u1; u += kKv4Warps) {
      const int key0 = u * kKv4Unit;
      const int next = u + kKv4Warps;
      float s[2][NT][4];
      kv4_scores<D, NT>(s[0], kk, 0, q);
      kv4_scores<D, NT>(s[1], kk, 1, q);
      if (next < u1)
        kk.load(k4, kscale, static_cast<long long>(next) * kKv4Unit, len - next * kKv4Unit, lane);
      if (key0 + kKv4Unit > all_see) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int lim = p.limit(row0 + nt * 8 + 2 * t + c, len) - key0 - g;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (16 * h >= lim) s[h][nt][c] = -INFINITY;
              if (16 * h + 8 >= lim) s[h][nt][2 + c] = -INFINITY;
            }
          }
      }
      // the reference a row's exponentials are taken against moves only when a score passes it
      // by more than 8 (log2 units): P stays below 2^8, and most units need no reduction
      bool grow = false;
      float mx[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          mx[nt][c] = fmaxf(fmaxf(s[0][nt][c], s[0][nt][2 + c]), fmaxf(s[1][nt][c], s[1][nt][2 + c])) * p.scale_log2;
          grow |= mx[nt][c] > m[nt][c] + 8.0f;
        }
      if (__any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float x = mx[nt][c];
            x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
            x = fmaxf(x, m[nt][c]);
            const float f = m[nt][c] == x ? 1.0f : ex2_approx(m[nt][c] - x);
            m[nt][c] = x;
            l[nt][c] *= f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              o[nt][i][c] *= f;
              o[nt][i][2 + c] *= f;
            }
          }
      }
      uint32_t pb[2][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float r0 = m[nt][0] == -INFINITY ? 0.0f : m[nt][0];
        const float r1 = m[nt][1] == -INFINITY ? 0.0f : m[nt][1];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float e[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) e[c] = ex2_approx(fmaf(s[h][nt][c], p.scale_log2, -((c & 1) ? r1 : r0)));
          l[nt][0] += e[0] + e[2];
          l[nt][1] += e[1] + e[3];
          pb[h][nt][0] = movmatrix(h2_bits(__floats2half2_rn(e[0], e[1])));
          pb[h][nt][1] = movmatrix(h2_bits(__floats2half2_rn(e[2], e[3])));
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const __half2 sa = bits_h2(__byte_perm(vv.vs[4 * h], vv.vs[4 * h + 1], 0x5410));
        const __half2 sb = bits_h2(__byte_perm(vv.vs[4 * h + 2], vv.vs[4 * h + 3], 0x5410));
#pragma unroll
        for (int w = 0; w < D / 64; ++w)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            // nibbles 4 half .. 4 half + 3 of two keys side by side, then expanded in key pairs
            const uint32_t sel = half ? 0x7632 : 0x5410;
            __half2 a[4], c[4];
            kv4_expand(__byte_perm(vv.v[4 * h][w], vv.v[4 * h + 1][w], sel), sa, a);
            kv4_expand(__byte_perm(vv.v[4 * h + 2][w], vv.v[4 * h + 3][w], sel), sb, c);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const int i = 4 * w + 2 * half;
              mma_f16(o[nt][i], h2_bits(a[0]), h2_bits(a[1]), h2_bits(c[0]), h2_bits(c[1]), pb[h][nt][0], pb[h][nt][1]);
              mma_f16(o[nt][i + 1], h2_bits(a[2]), h2_bits(a[3]), h2_bits(c[2]), h2_bits(c[3]), pb[h][nt][0],
                      pb[h][nt][1]);
            }
          }
      }
      if (next < u1)
        vv.load(v4, vscale, static_cast<long long>(next) * kKv4Unit, len - next * kKv4Unit, lane);
    }

    // ---- join the warps ----
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x = l[nt][c];
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 4);
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 8);
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 16);
        const int r = nt * 8 + 2 * t + c;
        if (g == 0) {
          sm.m[warp][r] = m[nt][c];
          sm.l[warp][r] = x;
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          *reinterpret_cast<float2*>(&sm.o[warp][r][g * (D / 8) + 2 * i]) = make_float2(o[nt][i][c], o[nt][i][2 + c]);
      }
    __syncthreads();
    const long long seg = static_cast<long long>(b) * per_b + in_b;
    const bool whole = u0 == 0 && u1 == n_units;
    for (int r = threadIdx.x; r < n_rows; r += kKv4Warps * 32) {
      float mm = sm.m[0][r];
#pragma unroll
      for (int w = 1; w < kKv4Warps; ++w) mm = fmaxf(mm, sm.m[w][r]);
      float ll = 0.0f;
#pragma unroll
      for (int w = 0; w < kKv4Warps; ++w) {
        // a warp that saw no key of this row has max -inf and sum 0
        const float f = sm.m[w][r] == -INFINITY ? 0.0f : ex2_approx(sm.m[w][r] - mm);
        sm.factor[w][r] = f;
        ll = fmaf(f, sm.l[w][r], ll);
      }
      sm.row_m[r] = mm;
      sm.row_l[r] = ll;
    }
    if (whole)
      for (int r = warp; r < n_rows; r += kKv4Warps) {
        const float off = kv4_offset<D>(p, bh, row0 + r, lane);
        if (lane == 0) sm.offset[r] = off;
      }
    __syncthreads();
    const long long out0 = bh * p.rows + row0;
    const long long slot = (blockIdx.x + seg) * kRows;
    for (int idx = threadIdx.x; idx < n_rows * (D / 2); idx += kKv4Warps * 32) {
      const int r = idx / (D / 2), ch = idx % (D / 2) * 2;
      float x = 0.0f, y = 0.0f;
#pragma unroll
      for (int w = 0; w < kKv4Warps; ++w) {
        const float2 v = *reinterpret_cast<const float2*>(&sm.o[w][r][ch]);
        x = fmaf(sm.factor[w][r], v.x, x);
        y = fmaf(sm.factor[w][r], v.y, y);
      }
      if (whole) {
        const float ll = sm.row_l[r];
        const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
        *reinterpret_cast<__half2*>(p.o + (out0 + r) * D + ch) = __floats2half2_rn(x * inv, y * inv);
      } else {
        *reinterpret_cast<float2*>(p.part_o + (slot + r) * D + ch) = make_float2(x, y);
      }
    }
    for (int r = threadIdx.x; r < n_rows; r += kKv4Warps * 32) {
      const float mm = sm.row_m[r], ll = sm.row_l[r];
      if (whole) {
        if (p.lse) p.lse[out0 + r] = kv4_lse(mm, ll, sm.offset[r]);
        if (p.weights) p.lse2[seg * kRows + r] = ll == 0.0f ? INFINITY : mm + log2f(ll);
      } else {
        p.part_ml[slot + r] = make_float2(mm, ll);
      }
    }
    if (!STREAM_K) return;
    // ---- next segment ----
    u_begin += u1 - u0;
    if (u_begin >= u_end) return;
    u0 = 0;
    if (++in_b == per_b) {
      in_b = 0;
      do {
        len = p.length(++b);
        n_units = kv4_units(len);
      } while (n_units == 0);
    }
    __syncthreads();   // the shared buffers are free again
  }
}

// Join the partials of a segment that several CTAs of the stream-K decode shared, and write
// the rows of sequences without a key. One CTA per (segment, row).
template <int D>
__global__ void __launch_bounds__(256) kv4_merge_kernel(Kv4Params p, int tile_rows) {
  __shared__ float so[8][D];
  __shared__ float sl[8];
  __shared__ float s_m, s_off;
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long seg = blockIdx.x;
  const long long per_b = static_cast<long long>(p.Hkv) * p.row_tiles;
  const int b = static_cast<int>(seg / per_b);
  const long long in_b = seg % per_b;
  const long long bh = static_cast<long long>(b) * p.Hkv + in_b / p.row_tiles;
  const int r = blockIdx.y, row = static_cast<int>(in_b % p.row_tiles) * tile_rows + r;
  if (row >= p.rows) return;
  const long long out = bh * p.rows + row;
  const int n_units = kv4_units(p.length(b));
  if (n_units == 0) {
    if (threadIdx.x < D) p.o[out * D + threadIdx.x] = __float2half_rn(0.0f);
    if (threadIdx.x == 0) {
      if (p.lse) p.lse[out] = -INFINITY;
      if (p.weights) p.lse2[seg * tile_rows + r] = INFINITY;
    }
    return;
  }
  const long long total = kv4_sum_units(p, p.B) * per_b;
  const long long ctas = total < p.ctas ? total : p.ctas;
  const long long t0 = kv4_sum_units(p, b) * per_b + in_b * n_units;
  // the CTA of unit u takes the range with u in [c total / ctas, (c + 1) total / ctas)
  const long long c0 = ((t0 + 1) * ctas - 1) / total, c1 = ((t0 + n_units) * ctas - 1) / total;
  if (c0 == c1) return;   // finished where it was computed
  float mm = -INFINITY;
  for (long long c = c0 + lane; c <= c1; c += 32) mm = fmaxf(mm, p.part_ml[(c + seg) * tile_rows + r].x);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xFFFFFFFFu, mm, d));
  float acc[D / 32], ll = 0.0f;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) acc[e] = 0.0f;
  for (long long c = c0 + warp; c <= c1; c += 8) {
    const long long at = (c + seg) * tile_rows + r;
    const float2 ml = p.part_ml[at];
    const float f = ml.x == -INFINITY ? 0.0f : ex2_approx(ml.x - mm);
    ll = fmaf(f, ml.y, ll);
#pragma unroll
    for (int e = 0; e < D / 32; ++e) acc[e] = fmaf(f, p.part_o[at * D + e * 32 + lane], acc[e]);
  }
#pragma unroll
  for (int e = 0; e < D / 32; ++e) so[warp][e * 32 + lane] = acc[e];
  if (lane == 0) sl[warp] = ll;
  if (warp == 0) {
    const float off = kv4_offset<D>(p, bh, row, lane);
    if (lane == 0) s_m = mm, s_off = off;
  }
  __syncthreads();
  ll = 0.0f;
#pragma unroll
  for (int w = 0; w < 8; ++w) ll += sl[w];
  if (threadIdx.x < D) {
    float x = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) x += so[w][threadIdx.x];
    p.o[out * D + threadIdx.x] = __float2half_rn(ll == 0.0f ? 0.0f : x / ll);
  }
  if (threadIdx.x == 0) {
    if (p.lse) p.lse[out] = kv4_lse(s_m, ll, s_off);
    if (p.weights) p.lse2[seg * tile_rows + r] = ll == 0.0f ? INFINITY : s_m + log2f(ll);
  }
}

// weights[b, h, key] += sum over the kv head's rows of softmax(scale * q K'^T)[row, key], from
// the rows' log-sum-exps that the decode left in lse2: the scores are computed again from the
// key codes (half of the cache's bytes), which needs no buffer of rows x keys scores. One warp
// per 32-key unit, each weight summed and stored by one lane: the same order every time.
template <int D>
__global__ void __launch_bounds__(kKv4Warps * 32) kv4_weights_kernel(Kv4Params p, int tile_rows) {
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const long long bh = blockIdx.y + static_cast<long long>(blockIdx.z) * gridDim.y;
  if (bh >= static_cast<long long>(p.B) * p.Hkv) return;
  const int len = p.length(static_cast<int>(bh / p.Hkv));
  const int all_see = p.causal ? max(0, len - p.Sq + 1) : len;
  const uint8_t* k4 = p.k4 + bh * p.cap * (D / 2);
  const __half* kscale = p.kscale + bh * p.cap * (D / 32);
  const int n_units = kv4_units(len);
  for (int u = blockIdx.x * kKv4Warps + warp; u < n_units; u += gridDim.x * kKv4Warps) {
    const int key0 = u * kKv4Unit;
    Kv4Keys<D> kk;
    kk.load(k4, kscale, key0, len - key0, lane);
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};   // keys g + 8 i
    for (int r0 = 0; r0 < p.rows; r0 += 8) {
      uint32_t q[1][D / 16][2];
      kv4_query<D>(q[0], p.q + (bh * p.rows + r0) * D, p.rows - r0, lane);
      float s[2][1][4];
      kv4_scores<D, 1>(s[0], kk, 0, q);
      kv4_scores<D, 1>(s[1], kk, 1, q);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = r0 + 2 * t + c;
        if (r >= p.rows) continue;
        const long long seg = bh * p.row_tiles + r / tile_rows;
        const float ref = p.lse2[seg * tile_rows + r % tile_rows];
        const int lim = (key0 + kKv4Unit > all_see ? p.limit(r, len) : len) - key0 - g;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (8 * i < lim) sum[i] += ex2_approx(fmaf(s[i / 2][0][2 * (i % 2) + c], p.scale_log2, -ref));
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], 1);
      sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], 2);
    }
    const float mine = t == 0 ? sum[0] : t == 1 ? sum[1] : t == 2 ? sum[2] : sum[3];
    const int key = key0 + g + 8 * t;
    if (key < len) p.weights[bh * p.cap + key] += mine;
  }
}

}  // namespace pasa
