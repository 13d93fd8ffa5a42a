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

constexpr int kEvictBins = 4096;

// One CTA per (sequence, kv head): the rows it keeps, ascending, -1 past the last. The
// threshold is found in three passes over the weights (read from L2 after the first), by their
// keys' bits 31 .. 20, 19 .. 10 and 9 .. 0: with 12 bits, weights of similar size spread over
// several counters even in the first pass. Zeros, the weight of every row not yet looked at,
// are counted by warp instead of one by one.
__global__ void __launch_bounds__(kEvictThreads) evict_select_kernel(const float* __restrict__ weights,
                                                                     const int* __restrict__ lengths,
                                                                     int* __restrict__ index, int Hkv, int Sk,
                                                                     long long cap, int budget, int recent) {
  __shared__ uint32_t hist[kEvictBins];
  __shared__ uint32_t s_warp[32], s_prefix, s_left;
  __shared__ int s_gt[32], s_eq[32];
  griddep_launch_dependents();
  const long long bh = blockIdx.x;
  const int len = lengths ? max(0, min(lengths[bh / Hkv], Sk)) : Sk;
  const float* w = weights + bh * cap;
  int* idx = index + bh * budget;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (len <= budget) {
    for (int j = tid; j < budget; j += kEvictThreads) idx[j] = j < len ? j : -1;
    return;
  }
  const int n = len - recent;           // candidates 0 .. n - 1
  uint32_t left = budget - recent;      // how many of them stay
  uint32_t prefix = 0;                  // the left-th largest candidate's key
  const bool any = left > 0;
  if (any) {
    constexpr uint32_t kZero = 0x80000000u;
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 20 : pass == 1 ? 10 : 0;
      const uint32_t mask = pass == 0 ? 0xFFFu : 0x3FFu;
      for (int i = tid; i < kEvictBins; i += kEvictThreads) hist[i] = 0;
      __syncthreads();
      for (int j0 = 0; j0 < n; j0 += 8 * kEvictThreads) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int j = j0 + i * kEvictThreads + tid;
          x[i] = j < n ? w[j] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t k = weight_key(x[i]);
          const bool in = j0 + i * kEvictThreads + tid < n &&
                          (pass == 0 || (k >> (pass == 1 ? 20 : 10)) == (prefix >> (pass == 1 ? 20 : 10)));
          const uint32_t zeros = __ballot_sync(0xFFFFFFFFu, in && k == kZero);
          if (in && k != kZero) atomicAdd(&hist[(k >> shift) & mask], 1u);
          if (zeros != 0 && lane == 0) atomicAdd(&hist[(kZero >> shift) & mask], static_cast<uint32_t>(__popc(zeros)));
        }
      }
      __syncthreads();
      // counters from the top, 4 to a thread: thread t has 4095 - 4 t .. 4092 - 4 t
      uint32_t c[4], sum = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[i] = hist[kEvictBins - 1 - 4 * tid - i];
        sum += c[i];
      }
      uint32_t before = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, before, d);
        if (lane >= d) before += x;
      }
      if (lane == 31) s_warp[warp] = before;
      __syncthreads();
      uint32_t below = lane < warp ? s_warp[lane] : 0;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) below += __shfl_xor_sync(0xFFFFFFFFu, below, d);
      before += below - sum;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (before < left && before + c[i] >= left) {   // one thread, one counter
          s_prefix = prefix | (static_cast<uint32_t>(kEvictBins - 1 - 4 * tid - i) << shift);
          s_left = left - before;
        }
        before += c[i];
      }
      __syncthreads();
      prefix = s_prefix;
      left = s_left;
      __syncthreads();
    }
  }
  // Each warp takes a run of rows: how many of its keys pass, and how many equal the threshold, of
  // which the first `left` in row order stay; then the row numbers.
  const int run = (len + 1023) / 1024 * 32;
  const int a = min(len, warp * run), e = min(len, a + run);
  int gt = 0, eq = 0;
  for (int j = a + lane; j < e; j += 32) {
    const uint32_t k = weight_key(w[j]);
    gt += j >= n || (any && k > prefix);
    eq += any && j < n && k == prefix;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    gt += __shfl_xor_sync(0xFFFFFFFFu, gt, d);
    eq += __shfl_xor_sync(0xFFFFFFFFu, eq, d);
  }
  if (lane == 0) s_gt[warp] = gt, s_eq[warp] = eq;
  __syncthreads();
  int gt_before = lane < warp ? s_gt[lane] : 0, eq_before = lane < warp ? s_eq[lane] : 0;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    gt_before += __shfl_xor_sync(0xFFFFFFFFu, gt_before, d);
    eq_before += __shfl_xor_sync(0xFFFFFFFFu, eq_before, d);
  }
  int eq_left = any ? static_cast<int>(left) - eq_before : 0;   // equal keys that still stay
  int pos = gt_before + min(eq_before, any ? static_cast<int>(left) : 0);
  const uint32_t lower = (1u << lane) - 1u;
  for (int j0 = a; j0 < e; j0 += 32) {
    const int j = j0 + lane;
    const uint32_t k = j < e ? weight_key(w[j]) : 0u;
    const bool same = j < e && any && j < n && k == prefix;
    const uint32_t m_same = __ballot_sync(0xFFFFFFFFu, same);
    const bool keep = (j < e && (j >= n || (any && k > prefix))) || (same && __popc(m_same & lower) < eq_left);
    const uint32_t m_keep = __ballot_sync(0xFFFFFFFFu, keep);
    if (keep) idx[pos + __popc(m_keep & lower)] = j;
    pos += __popc(m_keep);
    eq_left -= __popc(m_same);
  }
}

struct EvictPlanes {
  const unsigned char* src[kEvictPlanes + 1];
  unsigned char* dst[kEvictPlanes + 1];
  int row_bytes[kEvictPlanes + 1];
  int width[kEvictPlanes + 1];          // bytes of a row that a CTA moves
  int first_column[kEvictPlanes + 2];
  int n;                                // planes; entry n - 1 are the weights
};

// Move rows idx[r0 .. r1): N rows to a thread and round, `lanes` threads with a T each to a row.
// A round's rows are all read before any is written, and a row's old place is never before its new
// one, so in place a later round's rows are still there.
template <typename T>
__device__ __forceinline__ void move_rows(const unsigned char* src, unsigned char* dst, const int* idx, int row_bytes,
                                          int lanes, int r0, int r1, bool in_place) {
  constexpr int N = 8;
  const int per = kMoveThreads / lanes;   // rows of a block-wide step
  const int mine = threadIdx.x / lanes, at = threadIdx.x % lanes * static_cast<int>(sizeof(T));
  for (int base = r0; base < r1; base += per * N) {
    T x[N];
    int from[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = base + i * per + mine;
      from[i] = r < r1 ? idx[r] : -1;
      if (in_place && from[i] == r) from[i] = -1;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (from[i] >= 0) x[i] = *reinterpret_cast<const T*>(src + static_cast<long long>(from[i]) * row_bytes + at);
    if (in_place) __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (from[i] >= 0)
        *reinterpret_cast<T*>(dst + static_cast<long long>(base + i * per + mine) * row_bytes + at) = x[i];
    if (in_place) __syncthreads();
  }
}

// blockIdx.x: (sequence, kv head); blockIdx.y: a column of a plane's rows (a 32-byte sector in
// place, where only columns can move side by side; up to 128 bytes otherwise); blockIdx.z: a
// range of rows (all of them in place). The weights' CTAs also clear what is past the last row.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(EvictPlanes pl, const int* __restrict__ index,
                                                                  int* new_lengths, int Hkv, long long cap,
                                                                  long long out_cap, int budget, int rows_per_cta) {
  const long long bh = blockIdx.x;
  int p = 0;
  while (static_cast<int>(blockIdx.y) >= pl.first_column[p + 1]) ++p;
  const int col = (blockIdx.y - pl.first_column[p]) * pl.width[p];
  const int width = min(pl.width[p], pl.row_bytes[p] - col);
  const bool in_place = pl.src[p] == pl.dst[p];
  const unsigned char* src = pl.src[p] + bh * cap * pl.row_bytes[p] + col;
  unsigned char* dst = pl.dst[p] + bh * out_cap * pl.row_bytes[p] + col;
  const int r0 = blockIdx.z * rows_per_cta, r1 = min(budget, r0 + rows_per_cta);
  griddep_wait();
  const int* idx = index + bh * budget;
  if (pl.row_bytes[p] % 16 == 0)
    move_rows<uint4>(src, dst, idx, pl.row_bytes[p], width / 16, r0, r1, in_place);
  else if (pl.row_bytes[p] % 8 == 0)
    move_rows<uint2>(src, dst, idx, pl.row_bytes[p], width / 8, r0, r1, in_place);
  else
    move_rows<uint32_t>(src, dst, idx, pl.row_bytes[p], width / 4, r0, r1, in_place);
  if (p != pl.n - 1 || blockIdx.z != 0) return;
  // how many rows there are (all heads of a sequence keep as many), by the first -1
  int lo = 0, hi = budget;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (idx[mid] >= 0) lo = mid + 1; else hi = mid;
  }
  float* w = reinterpret_cast<float*>(dst);
  for (long long j = lo + static_cast<int>(threadIdx.x); j < out_cap; j += kMoveThreads) w[j] = 0.0f;
  if (new_lengths && bh % Hkv == 0 && threadIdx.x == 0) new_lengths[bh / Hkv] = lo;
}

}  // namespace pasa
