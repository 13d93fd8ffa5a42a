// Eviction from a key/value cache by accumulated attention weight: of each sequence longer than
// `budget` rows, every kv head keeps its last `recent` rows and, of the others, the rows with
// the largest weights (equal weights: the lowest row), in their old order.
//
// evict_select_kernel finds the rows (radix selection on the weights' bits), writes their
// numbers and the kept weights; evict_move_kernel moves the rows of every plane of the cache.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace pasa {

constexpr int kEvictThreads = 1024;
constexpr int kEvictPlanes = 8;     // planes of one cache
constexpr int kMoveThreads = 256;

// Weights as unsigned numbers in the same order: NaN counts as -inf, -0 as 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) w = -INFINITY;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One CTA per (sequence, kv head). weights and out_weights may be the same array.
__global__ void __launch_bounds__(kEvictThreads) evict_select_kernel(
    const float* weights, float* out_weights, const int* __restrict__ lengths, int* __restrict__ index, int Hkv, int Sk,
    long long cap, long long out_cap, int budget, int recent) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t s_prefix, s_left;
  __shared__ int s_gt[32], s_eq[32];
  griddep_launch_dependents();
  const long long bh = blockIdx.x;
  const int b = static_cast<int>(bh / Hkv);
  const int len = lengths ? max(0, min(lengths[b], Sk)) : Sk;
  const float* w = weights + bh * cap;
  float* ow = out_weights + bh * out_cap;
  int* idx = index + bh * budget;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int kept = min(len, budget);
  if (len <= budget) {
    for (int j = tid; j < budget; j += kEvictThreads) idx[j] = j < len ? j : -1;
    if (ow != w)
      for (int j = tid; j < len; j += kEvictThreads) ow[j] = w[j];
  } else {
    const int n = len - recent;          // candidates 0 .. n - 1
    uint32_t left = budget - recent;     // how many of them stay
    uint32_t prefix = 0, need_eq = 0;
    if (left > 0) {
      // the key of the left-th largest candidate, 8 bits at a time
      for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        for (int j = tid; j < n; j += kEvictThreads) {
          const uint32_t k = weight_key(w[j]);
          if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (warp == 0) {
          // bins from the top: lane l holds bins 255 - 8 l .. 248 - 8 l
          uint32_t c[8], sum = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            c[i] = hist[255 - 8 * lane - i];
            sum += c[i];
          }
          uint32_t before = sum;
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, before, d);
            if (lane >= d) before += x;
          }
          before -= sum;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (before < left && before + c[i] >= left) {
              s_prefix = prefix | (static_cast<uint32_t>(255 - 8 * lane - i) << shift);
              s_left = left - before;
            }
            before += c[i];
          }
        }
        __syncthreads();
        prefix = s_prefix;
        left = s_left;
        __syncthreads();
      }
      need_eq = left;
    }
    // in order: keys above the threshold, the first need_eq equal to it, the recent rows
    const bool any = budget > recent;
    int base = 0, base_eq = 0;
    for (int j0 = 0; j0 < len; j0 += kEvictThreads) {
      const int j = j0 + tid;
      const float x = j < len ? w[j] : 0.0f;
      const uint32_t k = weight_key(x);
      const bool eq = any && j < n && k == prefix;
      const bool gt = j < len && (j >= n || (any && k > prefix));
      const uint32_t m_eq = __ballot_sync(0xFFFFFFFFu, eq);
      if (lane == 0) s_eq[warp] = __popc(m_eq);
      __syncthreads();
      int eq_before = base_eq, eq_all = 0;
      for (int i = 0; i < 32; ++i) {
        if (i < warp) eq_before += s_eq[i];
        eq_all += s_eq[i];
      }
      eq_before += __popc(m_eq & ((1u << lane) - 1u));
      const bool keep = gt || (eq && eq_before < static_cast<int>(need_eq));
      const uint32_t m_keep = __ballot_sync(0xFFFFFFFFu, keep);
      if (lane == 0) s_gt[warp] = __popc(m_keep);
      __syncthreads();   // every weight of this round is read: it may be overwritten
      int pos = base, all = 0;
      for (int i = 0; i < 32; ++i) {
        if (i < warp) pos += s_gt[i];
        all += s_gt[i];
      }
      pos += __popc(m_keep & ((1u << lane) - 1u));
      if (keep) {
        idx[pos] = j;
        ow[pos] = x;
      }
      base += all;
      base_eq += eq_all;
    }
    __syncthreads();
  }
  for (long long j = kept + tid; j < out_cap; j += kEvictThreads) ow[j] = 0.0f;
}

struct EvictPlanes {
  const unsigned char* src[kEvictPlanes];
  unsigned char* dst[kEvictPlanes];
  int row_bytes[kEvictPlanes];
  int width[kEvictPlanes];          // bytes of a row that one thread moves
  int first_column[kEvictPlanes + 1];
  int n;
};

template <typename T, int N>
__device__ __forceinline__ void move_rows(const unsigned char* src, unsigned char* dst, const int* idx, int row_bytes,
                                          int r0, int r1, bool in_place) {
  // rows r0 .. r1, kMoveThreads * 4 at a time: all are read before any is written, and a row's
  // old place is never before its new one, so a later round's rows are still there
  for (int base = r0; base < r1; base += kMoveThreads * 4) {
    T x[4][N];
    int from[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = base + i * kMoveThreads + threadIdx.x;
      from[i] = r < r1 ? idx[r] : -1;
      if (from[i] == r && in_place) from[i] = -1;
      if (from[i] >= 0) {
        const T* s = reinterpret_cast<const T*>(src + static_cast<long long>(from[i]) * row_bytes);
#pragma unroll
        for (int e = 0; e < N; ++e) x[i][e] = s[e];
      }
    }
    if (in_place) __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = base + i * kMoveThreads + threadIdx.x;
      if (from[i] >= 0) {
        T* d = reinterpret_cast<T*>(dst + static_cast<long long>(r) * row_bytes);
#pragma unroll
        for (int e = 0; e < N; ++e) d[e] = x[i][e];
      }
    }
    if (in_place) __syncthreads();
  }
}

// blockIdx.x: (sequence, kv head); blockIdx.y: a column of a plane's rows, up to 32 bytes
// (a sector) wide; blockIdx.z: a range of rows (one range when rows move in place).
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(EvictPlanes pl,
                                                                  const int* __restrict__ index, int* new_lengths,
                                                                  int Hkv, long long cap, long long out_cap, int budget,
                                                                  int rows_per_cta) {
  const long long bh = blockIdx.x;
  const int b = static_cast<int>(bh / Hkv);
  griddep_wait();
  const int* idx = index + bh * budget;
  int p = 0;
  while (static_cast<int>(blockIdx.y) >= pl.first_column[p + 1]) ++p;
  const int col = (blockIdx.y - pl.first_column[p]) * pl.width[p];
  const bool in_place = pl.src[p] == pl.dst[p];
  const unsigned char* src = pl.src[p] + bh * cap * pl.row_bytes[p] + col;
  unsigned char* dst = pl.dst[p] + bh * out_cap * pl.row_bytes[p] + col;
  const int r0 = blockIdx.z * rows_per_cta, r1 = min(budget, r0 + rows_per_cta);
  switch (pl.width[p]) {
    case 32: move_rows<uint4, 2>(src, dst, idx, pl.row_bytes[p], r0, r1, in_place); break;
    case 16: move_rows<uint4, 1>(src, dst, idx, pl.row_bytes[p], r0, r1, in_place); break;
    case 8: move_rows<uint2, 1>(src, dst, idx, pl.row_bytes[p], r0, r1, in_place); break;
    default: move_rows<uint32_t, 1>(src, dst, idx, pl.row_bytes[p], r0, r1, in_place); break;
  }
  // the new length, by the head's last entry that is a row (all heads keep as many)
  if (new_lengths && bh % Hkv == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) {
    int lo = 0, hi = budget;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (idx[mid] >= 0) lo = mid + 1; else hi = mid;
    }
    new_lengths[b] = lo;
  }
}

}  // namespace pasa
