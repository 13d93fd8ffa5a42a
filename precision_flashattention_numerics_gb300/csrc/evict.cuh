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

constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kEvictPlanes = 8;     // planes of one cache
constexpr int kMoveThreads = 256;
constexpr int kEvictCluster = 4;    // CTAs of a (sequence, kv head), at most

// Weights as unsigned numbers in the same order: NaN counts as -inf, -0 as 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) w = -INFINITY;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kEvictBins = 2048;
constexpr int kEvictPer = 16;                               // weights of a thread
constexpr int kEvictChunk = kEvictThreads * kEvictPer;      // rows that a CTA holds in registers

// A cluster of CTAs per (sequence, kv head), each with an equal run of its rows: the rows the head
// keeps, ascending, -1 past the last: those with the budget largest keys, a recent row's key
// being above every weight's (kRecent) and that of a row past the last below (kNone). The
// threshold is found in three passes over the keys, by bits 31 .. 21, 20 .. 10 and 9 .. 0: with 11
// bits, weights of similar size spread over several counters even in the first pass. Zeros, the
// weight of every row not yet looked at, and recent rows are counted apart, not one by one in
// the same counter. Every CTA adds up the counters of all (distributed shared memory) and finds
// the same threshold. A CTA's first 8192 rows are read once and stay in registers; more are
// read again (from L2) in every pass, a chunk at a time.
__global__ void __launch_bounds__(kEvictThreads) evict_select_kernel(const float* __restrict__ weights,
                                                                     const int* __restrict__ lengths,
                                                                     int* __restrict__ index, int Hkv, int Sk,
                                                                     long long cap, int budget, int recent, int cluster) {
  __shared__ __align__(16) uint32_t hist[3][kEvictBins];
  __shared__ uint32_t s_warp[kEvictWarps], s_prefix, s_left;
  __shared__ int s_keep[kEvictWarps], s_eq[kEvictWarps];
  __shared__ float2 s_part;   // this CTA's keys above and equal to the threshold, as integers' bits
  griddep_launch_dependents();
  const long long bh = blockIdx.x / cluster;
  const int rank = blockIdx.x % cluster;
  const float* w = weights + bh * cap;
  int* idx = index + bh * budget;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int part = (Sk + cluster - 1) / cluster;   // rows of a CTA, by Sk: its loads wait for no length
  const int row0 = min(Sk, rank * part);
  const int chunks = (part + kEvictChunk - 1) / kEvictChunk;
  const int per = chunks > 1 ? kEvictPer : (part + kEvictThreads - 1) / kEvictThreads;   // elements of a lane
  uint32_t k[kEvictPer];                // element i: row `first` + 32 i of the chunk at hand
  const int first = row0 + warp * (32 * per) + lane;
  auto fetch = [&](int chunk) {   // the weights' bits, without branches between the loads
    const int base = chunk * kEvictChunk + first;
#pragma unroll
    for (int i = 0; i < kEvictPer; ++i) k[i] = __float_as_uint(__ldg(w + (i < per ? min(base + 32 * i, Sk - 1) : 0)));
  };
  fetch(0);
  const int len = lengths ? max(0, min(lengths[bh / Hkv], Sk)) : Sk;
  if (len <= budget) {   // all CTAs of the cluster
    for (int j = rank * kEvictThreads + tid; j < budget; j += cluster * kEvictThreads) idx[j] = j < len ? j : -1;
    return;
  }
  constexpr uint32_t kZero = 0x80000000u, kNone = 0u, kRecent = 0xFFFFFFFFu;
  uint32_t left = budget;               // of the keys that match `prefix` so far, how many stay
  uint32_t prefix = 0;                  // the budget-th largest key
  const int row1 = min(len, row0 + part);
  auto to_keys = [&](int chunk) {
    const int base = chunk * kEvictChunk + first;
#pragma unroll
    for (int i = 0; i < kEvictPer; ++i) {
      const int j = base + 32 * i;
      const uint32_t key = weight_key(__uint_as_float(k[i]));
      k[i] = i >= per || j >= row1 ? kNone : j >= len - recent ? kRecent : key;
    }
  };
  auto load = [&](int chunk) {
    fetch(chunk);
    to_keys(chunk);
  };
  to_keys(0);
  for (int i = tid; i < 3 * kEvictBins / 4; i += kEvictThreads) reinterpret_cast<uint4*>(hist[0])[i] = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const int fixed = pass == 1 ? 21 : 10;   // pass > 0: bits from here up are prefix's
    const uint32_t bins = pass == 2 ? 1024 : kEvictBins;
    int zeros = 0;
    for (int chunk = 0; chunk < chunks; ++chunk) {
      if (chunks > 1) load(chunk);
#pragma unroll
      for (int i = 0; i < kEvictPer; ++i) {
        zeros += k[i] == kZero;
        const bool in = 2u * k[i] + 2u > 2u;   // neither kNone nor kZero nor kRecent
        if (in && (pass == 0 || ((k[i] ^ prefix) >> fixed) == 0)) atomicAdd(&hist[pass][(k[i] >> shift) & (bins - 1)], 1u);
      }
    }
    zeros = __reduce_add_sync(0xFFFFFFFFu, zeros);
    if (lane == 0 && zeros > 0 && (pass == 0 || ((kZero ^ prefix) >> fixed) == 0))
      atomicAdd(&hist[pass][(kZero >> shift) & (bins - 1)], static_cast<uint32_t>(zeros));
    if (tid == 0 && rank == 0 && recent > 0 && (pass == 0 || ((kRecent ^ prefix) >> fixed) == 0))
      atomicAdd(&hist[pass][(kRecent >> shift) & (bins - 1)], static_cast<uint32_t>(recent));
    if (cluster > 1) cluster_sync_all(); else __syncthreads();
    // counters from the top, 4 to a thread: thread t has 2047 - 4 t .. 2044 - 4 t
    uint32_t c[4] = {0u, 0u, 0u, 0u};
    const uint32_t at = smem_u32(&hist[pass][kEvictBins - 4 - 4 * tid]);
    float4 x[kEvictCluster];   // all loads first
#pragma unroll
    for (int r = 0; r < kEvictCluster; ++r) {
      x[r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (r < cluster) x[r] = ld_cluster_float4(cluster > 1 ? mapa_shared(at, r) : at);
    }
#pragma unroll
    for (int r = 0; r < kEvictCluster; ++r) {
      c[0] += __float_as_uint(x[r].w), c[1] += __float_as_uint(x[r].z);
      c[2] += __float_as_uint(x[r].y), c[3] += __float_as_uint(x[r].x);
    }
    const uint32_t sum = c[0] + c[1] + c[2] + c[3];
    uint32_t before = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, before, d);
      if (lane >= d) before += x;
    }
    if (lane == 31) s_warp[warp] = before;
    __syncthreads();
    before += __reduce_add_sync(0xFFFFFFFFu, lane < warp ? s_warp[lane] : 0u) - sum;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (before < left && before + c[i] >= left) {   // one thread, one counter
        s_prefix = prefix | ((kEvictBins - 1 - 4 * tid - i) << shift);
        s_left = left - before;
      }
      before += c[i];
    }
    __syncthreads();
    prefix = s_prefix;
    left = s_left;
  }
  // Of the keys equal to the threshold the first `left` in row order stay. The CTA's counts and those
  // of the CTAs before it, then per chunk each warp's counts and the row numbers.
  int gt = 0, eq = 0;
  for (int chunk = 0; chunk < chunks; ++chunk) {
    if (chunks > 1) load(chunk);
#pragma unroll
    for (int i = 0; i < kEvictPer; ++i) {
      gt += k[i] > prefix;
      eq += k[i] == prefix;
    }
  }
  gt = __reduce_add_sync(0xFFFFFFFFu, gt);
  eq = __reduce_add_sync(0xFFFFFFFFu, eq);
  if (lane == 0) s_keep[warp] = gt, s_eq[warp] = eq;
  __syncthreads();
  if (cluster > 1 && warp == 0) {
    gt = __reduce_add_sync(0xFFFFFFFFu, lane < kEvictWarps ? s_keep[lane] : 0);
    eq = __reduce_add_sync(0xFFFFFFFFu, lane < kEvictWarps ? s_eq[lane] : 0);
    if (lane == 0) s_part = make_float2(__int_as_float(gt), __int_as_float(eq));
  }
  int pos0 = 0, eq_left0 = static_cast<int>(left);   // before the chunk
  if (cluster > 1) {
    cluster_sync_all();
    // lane r has CTA r's
    float2 x = make_float2(0.0f, 0.0f);
    if (lane < rank) x = ld_cluster_float2(mapa_shared(smem_u32(&s_part), lane));
    const int eq_ranks = __reduce_add_sync(0xFFFFFFFFu, __float_as_int(x.y));
    pos0 = __reduce_add_sync(0xFFFFFFFFu, __float_as_int(x.x)) + min(eq_ranks, eq_left0);
    eq_left0 = max(0, eq_left0 - eq_ranks);
  }
  for (int chunk = 0; chunk < chunks; ++chunk) {
    const int base = chunk * kEvictChunk + first;
    if (chunks > 1) {
      load(chunk);
      gt = 0, eq = 0;
#pragma unroll
      for (int i = 0; i < kEvictPer; ++i) {
        gt += k[i] > prefix;
        eq += k[i] == prefix;
      }
      gt = __reduce_add_sync(0xFFFFFFFFu, gt);
      eq = __reduce_add_sync(0xFFFFFFFFu, eq);
      __syncthreads();   // the counts before are read
      if (lane == 0) s_keep[warp] = gt, s_eq[warp] = eq;
      __syncthreads();
    }
    const int gt_warp = lane < kEvictWarps ? s_keep[lane] : 0, eq_warp = lane < kEvictWarps ? s_eq[lane] : 0;
    const int gt_before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? gt_warp : 0);
    const int eq_before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? eq_warp : 0);
    const int gt_all = __reduce_add_sync(0xFFFFFFFFu, gt_warp), eq_all = __reduce_add_sync(0xFFFFFFFFu, eq_warp);
    int pos = pos0 + gt_before + min(eq_before, eq_left0);
    int eq_left = max(0, eq_left0 - eq_before);
    const uint32_t lower = (1u << lane) - 1u;
#pragma unroll
    for (int i = 0; i < kEvictPer; ++i) {
      bool keep = k[i] > prefix;
      const uint32_t same = __ballot_sync(0xFFFFFFFFu, k[i] == prefix);
      if (same != 0) {
        keep |= k[i] == prefix && __popc(same & lower) < eq_left;
        eq_left = max(0, eq_left - __popc(same));
      }
      const uint32_t kept = __ballot_sync(0xFFFFFFFFu, keep);
      if (keep) idx[pos + __popc(kept & lower)] = base + 32 * i;
      pos += __popc(kept);
    }
    pos0 += gt_all + min(eq_all, eq_left0);
    eq_left0 = max(0, eq_left0 - eq_all);
  }
  if (cluster > 1) cluster_sync_all();   // no CTA ends while another reads its counters
}

struct EvictPlanes {
  const unsigned char* src[kEvictPlanes + 1];
  unsigned char* dst[kEvictPlanes + 1];
  int row_bytes[kEvictPlanes + 1];
  int width[kEvictPlanes + 1];          // bytes of a row that a CTA moves: a column
  int parts[kEvictPlanes + 1];          // CTAs of a column: each the rows of a round (in place one has all)
  int first[kEvictPlanes + 2];          // blockIdx.y of a plane's first CTA
  int n;                                // planes; entry n - 1 are the weights
};

// The word that a thread moves, and the rows that a CTA moves in a round.
__host__ __device__ constexpr int move_word(int row_bytes) { return row_bytes % 16 == 0 ? 16 : row_bytes % 8 == 0 ? 8 : 4; }
__host__ __device__ constexpr int move_rows_per_round(int row_bytes, int width) {
  return kMoveThreads / ((width < row_bytes ? width : row_bytes) / move_word(row_bytes)) * 4;
}

// Move rows idx[r0 .. r1): 4 rows to a thread and round, `lanes` threads with a T each to a row.
// A round's rows are all read before any is written, and a row's old place is never before its new
// one, so in place a later round's rows are still there.
template <typename T>
__device__ __forceinline__ void move_rows(const unsigned char* src, unsigned char* dst, const int* idx, int row_bytes,
                                          int lanes, int r0, int r1, bool in_place) {
  constexpr int N = 4;
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

// blockIdx.x: (sequence, kv head); blockIdx.y: a part of a column of a plane's rows (a column is a
// 32-byte sector in place, where only columns can move side by side; up to 128 bytes otherwise).
// The weights' first CTA also clears what is past the last row. `index` is not __restrict__: the selection
// writes it while this kernel already runs, so its loads must not count as those of constants, which
// may go through the read-only cache or ahead of griddep_wait().
__global__ void __launch_bounds__(kMoveThreads, 6) evict_move_kernel(EvictPlanes pl, const int* index, int* new_lengths,
                                                                     int Hkv, long long cap, long long out_cap,
                                                                     int budget) {
  const long long bh = blockIdx.x;
  int p = 0;
  while (static_cast<int>(blockIdx.y) >= pl.first[p + 1]) ++p;
  const int row_bytes = pl.row_bytes[p];
  const int column = (blockIdx.y - pl.first[p]) / pl.parts[p], part = blockIdx.y - pl.first[p] - column * pl.parts[p];
  const int col = column * pl.width[p];
  const int width = min(pl.width[p], row_bytes - col);
  const bool in_place = pl.src[p] == pl.dst[p];
  const unsigned char* src = pl.src[p] + bh * cap * row_bytes + col;
  unsigned char* dst = pl.dst[p] + bh * out_cap * row_bytes + col;
  const int word = move_word(row_bytes);
  const int lanes = width / word;
  const int* idx = index + bh * budget;
  const int rows = pl.parts[p] == 1 ? budget : move_rows_per_round(row_bytes, pl.width[p]);
  const int a = part * rows, b = min(budget, a + rows);   // budget <= INT_MAX - 65536
  griddep_wait();
  if (word == 16)
    move_rows<uint4>(src, dst, idx, row_bytes, lanes, a, b, in_place);
  else if (word == 8)
    move_rows<uint2>(src, dst, idx, row_bytes, lanes, a, b, in_place);
  else
    move_rows<uint32_t>(src, dst, idx, row_bytes, lanes, a, b, in_place);
  if (p != pl.n - 1 || part != 0) return;
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
