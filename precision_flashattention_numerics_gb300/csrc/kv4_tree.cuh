// Attention for drafted tokens over the 4-bit cache of kv4_store.cuh: the query rows of a sequence are the nodes of a tree
// (several guesses of what comes next); each sees the cache's rows, its ancestors and itself. The nodes' own
// keys and values are fp16 and not in the cache yet.
//
// With g heads to a kv head and n nodes a kv head has g n query rows, tens to hundreds, against every cached row: too
// many for kv4_decode_kernel, whose 8 or 16 rows are one side of a mma.sync and which would read and expand the cache once
// for each of them. Here 128 rows are the M side of tcgen05.mma, and a cached row is expanded to fp16 once for all of them.
//
// One CTA works on a segment (sequence, kv head, tile of 128 rows), 128 keys at a time. 16 warps:
//   0-3   softmax and epilogue, a thread to a row (TMEM lane)
//   4     brings codes to shared memory (cp.async.bulk), kRaw blocks ahead
//   5, 6  issue S = Q K'^T and O += P V
//   8-15  expand codes to fp16 K' and V tiles in the MMA's swizzled layout
// Codes are expanded to s c, which fp16 holds exactly. A word of 8 codes gives the channel order 0, 4, 1, 5, 2, 6, 3, 7 without
// a shuffle; Q is brought to that order when it goes to TMEM, and the epilogue puts O's columns back. Q and P are
// A operands in TMEM. Scores, maxima, sums and O are fp32, P is rounded to fp16 (2^-11).
// Registers: the softmax holds a row's 128 scores, so its warps take what the others leave (setmaxnreg:
// 208 + 56 + 2 x 120 <= 4 x 128 a thread).
//
// Items. A segment is a list of key blocks: first the nodes, then the cache's blocks from its last, partial one
// on. (What is read without the ring, nodes and the partial block, comes first, while the ring fills.)
//
// Work split. The segments' items are numbered in order, a segment's start counting as kTreeStart items, and CTA c takes the
// c-th of equal ranges: uneven lengths keep all SMs equally busy. A segment inside one CTA is finished there, else
// its CTAs leave (O, max, sum) partials that kv4_tree_merge_kernel joins.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "attn_fwd.cuh"
#include "kv4_store.cuh"
#include "ptx.cuh"

namespace pasa {
namespace tree {

constexpr int kThreads = 512;
constexpr int kRows = 128;       // of a tile
constexpr int kKeys = 128;       // of a block
constexpr int kMaxNodes = 128;
constexpr int kStages = 2;       // of expanded tiles
constexpr int kRaw = 4;          // of codes
constexpr int kCtas = 152;
constexpr int kStart = 2;        // items that the start and end of a segment cost
constexpr int kExpandThreads = 256;

struct Params {
  const __half *q, *k, *v;       // [B, Hq, Sq, D], [B, Hkv, Sq, D]: the nodes
  const int *parents;            // [B, Sq] or nullptr: a chain
  const int *counts;             // [B] or nullptr: Sq nodes in every sequence
  const uint8_t *k4, *v4;
  const __half *kscale, *vscale, *shift;
  const int* lengths;            // [B] or nullptr: Sk rows in every sequence
  __half* o;
  float* lse;
  float* part_o;                 // [2 CTAs][D / 4][rows][4]: a CTA's first segment, and its last
  float2* part_ml;               // [2 CTAs][rows]: max (log2 units), sum
  int B, Hkv, Sq, rows, row_tiles;
  int Sk, cap, ctas;
  float scale, scale_log2;

  __device__ __forceinline__ int length(int b) const {
    return lengths ? min(max(lengths[b], 0), Sk) : Sk;
  }
  __device__ __forceinline__ int count(int b) const { return counts ? min(max(counts[b], 0), Sq) : Sq; }
  // Key blocks of a segment, and what it weighs in the shares; 0 without a node.
  __device__ __forceinline__ int items(int b) const { return count(b) == 0 ? 0 : 1 + (length(b) + kKeys - 1) / kKeys; }
  __device__ __forceinline__ int weight(int b) const {
    const int n = items(b);
    return n == 0 ? 0 : n + kStart;
  }
};

// A CTA's range of the items of all segments, and the segments in it, one after another. Made and advanced
// by whole warps.
struct Range {
  const Params& p;
  int todo, b, in_b, r0, n_items, per_b;
  int j0, j1;      // items of the segment at hand
  bool first;      // it is the CTA's first

  // The sum of the weights of sequences 0 .. b_end - 1.
  static __device__ __forceinline__ int sum(const Params& p, int b_end) {
    int n = 0;
    for (int b = threadIdx.x & 31; b < b_end; b += 32) n += p.weight(b);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, d);
    return n;
  }
  static __device__ __forceinline__ int first_of(int total, int ctas, int c) {
    const int base = total / ctas, more = total - base * ctas;
    return c * base + min(c, more);
  }
  static __device__ __forceinline__ int cta_of(int total, int ctas, int u) {
    const int base = total / ctas, more = total - base * ctas, split = more * (base + 1);
    return u < split ? u / (base + 1) : more + (u - split) / base;
  }
  __device__ __forceinline__ Range(const Params& params) : p(params), todo(0), first(true) {
    per_b = p.Hkv * p.row_tiles;
    const int total = sum(p, p.B) * per_b;
    const int ctas = min(total, p.ctas);
    if (static_cast<int>(blockIdx.x) >= ctas) return;
    int place = first_of(total, ctas, blockIdx.x);
    todo = first_of(total, ctas, blockIdx.x + 1) - place;
    // the sequence that the range starts in: 32 at a time
    const int lane = threadIdx.x & 31;
    for (int b0 = 0;; b0 += 32) {
      const int w = b0 + lane < p.B ? p.weight(b0 + lane) * per_b : 0;
      int upto = w;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, upto, d);
        if (lane >= d) upto += x;
      }
      const uint32_t past = __ballot_sync(0xFFFFFFFFu, upto > place);
      if (past != 0) {
        const int l = __ffs(past) - 1;
        place -= __shfl_sync(0xFFFFFFFFu, upto - w, l);
        b = b0 + l;
        break;
      }
      place -= __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
    n_items = p.items(b);
    in_b = place / (n_items + kStart);
    r0 = place - in_b * (n_items + kStart) - kStart;
  }
  // The next segment with items; false at the end of the range.
  __device__ __forceinline__ bool next() {
    if (todo <= 0) return false;
    const int r1 = min(n_items, r0 + todo);
    todo -= r1 - r0;
    j0 = max(0, r0);
    j1 = r1;
    return j1 > j0;   // else the range ends in what a segment's start weighs
  }
  __device__ __forceinline__ void advance() {
    first = false;
    r0 = -kStart;
    if (todo > 0 && ++in_b == per_b) {
      in_b = 0;
      do {
        n_items = p.items(++b);
      } while (n_items == 0);
    }
  }
  __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == n_items; }
  __device__ __forceinline__ long long head() const { return static_cast<long long>(b) * p.Hkv + in_b / p.row_tiles; }
  __device__ __forceinline__ int row0() const { return in_b % p.row_tiles * kRows; }
};

template <int D>
struct Smem {
  static constexpr int kTile = kKeys * D * 2;
  static constexpr int kChunk = kKeys * 128;      // one 64-channel column of a tile
  static constexpr int kCodes = kKeys * D / 2;
  alignas(1024) uint8_t k[kStages][kTile];
  alignas(1024) uint8_t v[kStages][kTile];
  alignas(128) uint8_t raw[kRaw][2][kCodes];
  uint64_t raw_full[kRaw], raw_empty[kRaw];       // codes have landed; all expanding warps have read them
  uint64_t k_full[kStages], k_empty[kStages];     // expanded (8 warps); QK done
  uint64_t v_full[kStages], v_empty[kStages];
  uint64_t q_full;                                // Q of a segment is in TMEM (4 warps)
  uint64_t s_full[2], s_free[2];
  uint64_t p_full, p_free;
  uint64_t drain[2];
  uint32_t tmem_base;
  int abort_flag;
};

template <int D>
struct Tmem {
  __host__ __device__ static constexpr int s(int b) { return b * kKeys; }
  static constexpr int o = 2 * kKeys;
  static constexpr int p = o + D;
  static constexpr int q = p + kKeys / 2;
  static_assert(q + D / 2 <= 512, "TMEM budget");
};

template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// 8 channels of a 16-byte unit in the order 0, 4, 1, 5, 2, 6, 3, 7, kv4_expand's.
__device__ __forceinline__ uint4 code_order(uint4 x) {
  return make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632), __byte_perm(x.y, x.w, 0x5410),
                    __byte_perm(x.y, x.w, 0x7632));
}
// The channel of a column of O.
__host__ __device__ constexpr int channel_of(int col) { return (col & ~7) + (col & 1) * 4 + (col & 7) / 2; }
__host__ __device__ constexpr int column_of(int ch) { return (ch & ~7) + (ch & 3) * 2 + (ch & 7) / 4; }

// 32 channels (group w of a row) of codes, expanded into a tile. Lanes of groups 2 and 3 write their units in another
// order than those of 0 and 1, whose 64-channel column lies in the same banks.
template <int D>
__device__ __forceinline__ void put_codes(uint8_t* tile, int row, int w, uint4 codes, __half scale) {
  const __half2 s2 = __half2half2(scale);
  const bool other = D == 128 && (w & 2);
  const uint32_t in[4] = {other ? codes.z : codes.x, other ? codes.w : codes.y, other ? codes.x : codes.z, other ? codes.y : codes.w};
  uint8_t* at = tile + (w >> 1) * Smem<D>::kChunk + row * 128;
  const int x = ((w & 1) * 4) ^ (row & 7) ^ (other ? 2 : 0);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __half2 h[4];
    kv4_expand(in[i], s2, h);
    *reinterpret_cast<uint4*>(at + ((x ^ i) * 16)) = make_uint4(h2_bits(h[0]), h2_bits(h[1]), h2_bits(h[2]), h2_bits(h[3]));
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv4_tree_kernel(const __grid_constant__ Params p) {
  using S = Smem<D>;
  using TM = Tmem<D>;
  static_assert(sizeof(S) + 1024 <= 227 * 1024, "shared memory per CTA");
  extern __shared__ uint8_t smem_raw[];
  S& s = *reinterpret_cast<S*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  griddep_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < kRaw; ++i) { mbar_init(&s.raw_full[i], 1); mbar_init(&s.raw_empty[i], 8); }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s.k_full[i], 8);
      mbar_init(&s.k_empty[i], 1);
      mbar_init(&s.v_full[i], 8);
      mbar_init(&s.v_empty[i], 1);
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.s_free[i], 4);
    }
    mbar_init(&s.q_full, 4);
    mbar_init(&s.p_full, 4);
    mbar_init(&s.p_free, 1);
    mbar_init(&s.drain[0], 1);
    mbar_init(&s.drain[1], 1);
    s.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 5) {
    tmem_alloc(&s.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  volatile int* abort_flag = &s.abort_flag;
  Range seg(p);

  if (warp >= 8) {
    // ------------------------------------------------------------------ codes to fp16
    regs_down<120>();
    const int t = tid - 256;
    constexpr int kGroups = D / 32;                              // 16-byte chunks of a row of codes
    constexpr int kPer = kKeys * kGroups / kExpandThreads;       // of a tile, for a thread
    const int w = t % kGroups, row_t = t / kGroups;
    constexpr int kRowStep = kExpandThreads / kGroups;
    int it = 0, rc = 0;   // items and ring blocks so far
    bool ok = true;
    auto tile_free = [&](uint64_t* empty) {
      return it < kStages || mbar_wait(&empty[it % kStages], (it / kStages - 1) & 1, abort_flag, 0x2101);
    };
    auto tile_done = [&](uint64_t* full) {
      fence_proxy_async_smem();   // the MMA reads the tile through the async proxy
      __syncwarp();
      mbar_arrive_if(&full[it % kStages], lane == 0);
    };
    while (ok && seg.next()) {
      const long long bh = seg.head();
      const int len = p.length(seg.b), n_blocks = seg.n_items - 1;
      const long long plane = bh * p.cap;
      // scales of a block's chunks, asked for a block ahead
      __half ks[kPer], vs[kPer];
      auto ask_scales = [&](int j) {
        const long long row = plane + static_cast<long long>(n_blocks - j) * kKeys + row_t;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          ks[i] = p.kscale[(row + i * kRowStep) * kGroups + w];
          vs[i] = p.vscale[(row + i * kRowStep) * kGroups + w];
        }
      };
      auto in_ring = [&](int j) { return j >= 2 || (j == 1 && len % kKeys == 0); };
      if (in_ring(seg.j0)) ask_scales(seg.j0);
      for (int j = seg.j0; j < seg.j1; ++j, ++it) {
        uint8_t* kt = s.k[it % kStages];
        uint8_t* vt = s.v[it % kStages];
        if (in_ring(j)) {
          __half k_now[kPer], v_now[kPer];
#pragma unroll
          for (int i = 0; i < kPer; ++i) k_now[i] = ks[i], v_now[i] = vs[i];
          if (j + 1 < seg.j1) ask_scales(j + 1);
          const int slot = rc % kRaw;
          if (!mbar_wait(&s.raw_full[slot], (rc / kRaw) & 1, abort_flag, 0x2102)) { ok = false; break; }
          if (!tile_free(s.k_empty)) { ok = false; break; }
          uint4 codes[2][kPer];
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            codes[0][i] = *reinterpret_cast<const uint4*>(s.raw[slot][0] + (t + i * kExpandThreads) * 16);
            codes[1][i] = *reinterpret_cast<const uint4*>(s.raw[slot][1] + (t + i * kExpandThreads) * 16);
          }
#pragma unroll
          for (int i = 0; i < kPer; ++i) put_codes<D>(kt, row_t + i * kRowStep, w, codes[0][i], k_now[i]);
          tile_done(s.k_full);
          mbar_arrive_if(&s.raw_empty[slot], lane == 0);   // after tile_done's __syncwarp: every lane has its codes
          if (!tile_free(s.v_empty)) { ok = false; break; }
#pragma unroll
          for (int i = 0; i < kPer; ++i) put_codes<D>(vt, row_t + i * kRowStep, w, codes[1][i], v_now[i]);
          tile_done(s.v_full);
          ++rc;
        } else if (j == 1) {
          // the cache's last block, with fewer than 128 rows: nothing past the last is read
          const int row0 = (n_blocks - 1) * kKeys, n = len - row0;
          uint4 codes[2][kPer];
          __half sc[2][kPer];
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const int r = row_t + i * kRowStep;
            const long long at = plane + row0 + r;
            codes[0][i] = codes[1][i] = make_uint4(0u, 0u, 0u, 0u);
            sc[0][i] = sc[1][i] = __ushort_as_half(0);
            if (r < n) {
              codes[0][i] = *reinterpret_cast<const uint4*>(p.k4 + at * (D / 2) + w * 16);
              codes[1][i] = *reinterpret_cast<const uint4*>(p.v4 + at * (D / 2) + w * 16);
              sc[0][i] = p.kscale[at * kGroups + w];
              sc[1][i] = p.vscale[at * kGroups + w];
            }
          }
          if (j + 1 < seg.j1) ask_scales(j + 1);
          if (!tile_free(s.k_empty)) { ok = false; break; }
#pragma unroll
          for (int i = 0; i < kPer; ++i) put_codes<D>(kt, row_t + i * kRowStep, w, codes[0][i], sc[0][i]);
          tile_done(s.k_full);
          if (!tile_free(s.v_empty)) { ok = false; break; }
#pragma unroll
          for (int i = 0; i < kPer; ++i) put_codes<D>(vt, row_t + i * kRowStep, w, codes[1][i], sc[1][i]);
          tile_done(s.v_full);
        } else {
          // the nodes: K - shift and V in fp16, rows past the last node 0
          const int n = p.count(seg.b);
          const __half* kp = p.k + bh * p.Sq * D;
          const __half* vp = p.v + bh * p.Sq * D;
          constexpr int kUnits = D / 8, kTurns = kKeys * kUnits / kExpandThreads;
          const int u = t % kUnits, r0 = t / kUnits;
          constexpr int kStep = kExpandThreads / kUnits;
          uint4 sh = make_uint4(0u, 0u, 0u, 0u);
          if (p.shift) sh = *reinterpret_cast<const uint4*>(p.shift + bh * D + u * 8);
          if (in_ring(j + 1) && j + 1 < seg.j1) ask_scales(j + 1);
          if (!tile_free(s.k_empty) || !tile_free(s.v_empty)) { ok = false; break; }
#pragma unroll
          for (int i = 0; i < kTurns; ++i) {
            const int r = r0 + i * kStep;
            uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
            if (r < n) {
              x = *reinterpret_cast<const uint4*>(kp + r * D + u * 8);
              y = *reinterpret_cast<const uint4*>(vp + r * D + u * 8);
              x = make_uint4(hsub2_rn(x.x, sh.x), hsub2_rn(x.y, sh.y), hsub2_rn(x.z, sh.z), hsub2_rn(x.w, sh.w));
            }
            const int off = (u / 8) * S::kChunk + r * 128 + (((u % 8) ^ (r & 7)) * 16);
            *reinterpret_cast<uint4*>(kt + off) = code_order(x);
            *reinterpret_cast<uint4*>(vt + off) = code_order(y);
          }
          tile_done(s.k_full);
          tile_done(s.v_full);
        }
      }
      seg.advance();
    }
  } else if (warp >= 4) {
    regs_down<56>();
    if (warp == 4) {
      // ---------------------------------------------------------------- the ring of codes
      int rc = 0;
      bool ok = true;
      while (ok && seg.next()) {
        const long long plane = seg.head() * p.cap;
        const int n_blocks = seg.n_items - 1;
        const int from = p.length(seg.b) % kKeys == 0 ? 1 : 2;   // items before are not read through the ring
        for (int j = max(seg.j0, from); j < seg.j1; ++j, ++rc) {
          const int slot = rc % kRaw;
          if (rc >= kRaw && !mbar_wait(&s.raw_empty[slot], (rc / kRaw - 1) & 1, abort_flag, 0x2201)) { ok = false; break; }
          if (lane == 0) {
            const long long at = (plane + static_cast<long long>(n_blocks - j) * kKeys) * (D / 2);
            mbar_arrive_expect_tx(&s.raw_full[slot], 2 * S::kCodes);
            bulk_load_1d(s.raw[slot][0], p.k4 + at, S::kCodes, &s.raw_full[slot]);
            bulk_load_1d(s.raw[slot][1], p.v4 + at, S::kCodes, &s.raw_full[slot]);
          }
          __syncwarp();
        }
        seg.advance();
      }
      if (*abort_flag) {   // let the copies land before the shared memory goes away
        const uint64_t t0 = globaltimer_ns();
        for (int c = max(0, rc - kRaw); c < rc; ++c)
          while (!mbar_try_wait(&s.raw_full[c % kRaw], (c / kRaw) & 1) && globaltimer_ns() - t0 < kWaitTimeoutNs) {
          }
      }
    } else if (warp == 5) {
      // ---------------------------------------------------------------- S = Q K'^T
      constexpr uint32_t id_s = idesc_f16(kRows, kKeys, true, false);
      constexpr uint32_t hi = sdesc_hi_sw128(1024);
      const uint32_t k_lo = sdesc_lo(smem_u32(s.k[0]), 16);
      int it = 0, nth = 0;
      bool ok = true;
      while (ok && seg.next()) {
        if (!mbar_wait(&s.q_full, nth & 1, abort_flag, 0x2301)) break;
        for (int j = seg.j0; j < seg.j1; ++j, ++it) {
          const int st = it % kStages, sb = it & 1;
          if (!mbar_wait(&s.k_full[st], (it / kStages) & 1, abort_flag, 0x2302)) { ok = false; break; }
          if (it >= 2 && !mbar_wait(&s.s_free[sb], ((it >> 1) - 1) & 1, abort_flag, 0x2303)) { ok = false; break; }
          tc_fence_after();
          if (lane == 0) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_ts_w(tmem + TM::s(sb), tmem + TM::q + kk * 8,
                       k_lo + ((st * S::kTile + (kk / 4) * S::kChunk + (kk % 4) * 32) >> 4), hi, id_s, kk > 0 ? 1u : 0u);
            mma_commit(&s.s_full[sb]);
            mma_commit(&s.k_empty[st]);
          }
          __syncwarp();
        }
        ++nth;
        seg.advance();
      }
      if (lane == 0) {   // every MMA done before TMEM is given back
        mma_commit(&s.drain[0]);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(&s.drain[0], 0) && globaltimer_ns() - t0 < kWaitTimeoutNs) {
        }
      }
    } else if (warp == 6) {
      // ---------------------------------------------------------------- O += P V
      constexpr uint32_t id_o = idesc_f16(kRows, D, true, true);
      constexpr uint32_t hi = sdesc_hi_sw128(1024);
      const uint32_t v_lo = sdesc_lo(smem_u32(s.v[0]), S::kChunk);
      int it = 0;
      bool ok = true;
      while (ok && seg.next()) {
        for (int j = seg.j0; j < seg.j1; ++j, ++it) {
          const int st = it % kStages;
          if (!mbar_wait(&s.v_full[st], (it / kStages) & 1, abort_flag, 0x2401)) { ok = false; break; }
          if (!mbar_wait(&s.p_full, it & 1, abort_flag, 0x2402)) { ok = false; break; }
          tc_fence_after();
          if (lane == 0) {
            const uint32_t more = j > seg.j0 ? 1u : 0u;
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
              mma_ts_w(tmem + TM::o, tmem + TM::p + kk * 8, v_lo + ((st * S::kTile + kk * 2048) >> 4), hi, id_o, kk > 0 ? 1u : more);
            mma_commit(&s.p_free);
            mma_commit(&s.v_empty[st]);
          }
          __syncwarp();
        }
        seg.advance();
      }
      if (lane == 0) {
        mma_commit(&s.drain[1]);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(&s.drain[1], 0) && globaltimer_ns() - t0 < kWaitTimeoutNs) {
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ softmax + epilogue
    regs_up<208>();
    const int r = tid;
    const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t tO = tmem + lane_base + TM::o, tP = tmem + lane_base + TM::p, tQ = tmem + lane_base + TM::q;
    const float sl2 = p.scale_log2;
    constexpr int kPairs = kKeys / 2;
    int it = 0;
    bool ok = true;
    while (ok && seg.next()) {
      const long long bh = seg.head();
      const int row = seg.row0() + r;
      const int len = p.length(seg.b), n_blocks = seg.n_items - 1, nodes = p.count(seg.b);
      const int node = row % p.Sq;
      const bool live = row < p.rows && node < nodes;
      const bool any_live = __any_sync(0xFFFFFFFFu, live);   // a warp without one only keeps the barriers going
      // Q to TMEM; the QKs of the segment before are done, as this warp has seen the last one's scores
      float offset = 0.0f;
      if (any_live) {
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (bh * p.rows + row) * D);
        const uint4* sh = p.shift && p.lse ? reinterpret_cast<const uint4*>(p.shift + bh * D) : nullptr;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (live) x = __ldg(src + c * 4 + i);
            if (sh) {
              const uint4 y = __ldg(sh + c * 4 + i);
              const uint32_t xa[4] = {x.x, x.y, x.z, x.w}, ya[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 a = __half22float2(bits_h2(xa[e])), m = __half22float2(bits_h2(ya[e]));
                offset = fmaf(a.x, m.x, fmaf(a.y, m.y, offset));
              }
            }
            x = code_order(x);
            w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
          }
          tmem_st_x16(tQ + c * 16, w);
        }
        tmem_st_wait();
      }
      tc_fence_before();
      __syncwarp();
      mbar_arrive_if(&s.q_full, lane == 0);
      // the nodes that this row's node sees
      uint32_t see[kMaxNodes / 32] = {0u, 0u, 0u, 0u};
      if (live && seg.j0 == 0) {
        if (p.parents) {
          const int* up = p.parents + static_cast<long long>(seg.b) * p.Sq;
          for (int i = node; i >= 0;) {
#pragma unroll
            for (int e = 0; e < kMaxNodes / 32; ++e)
              if (i >> 5 == e) see[e] |= 1u << (i & 31);
            const int next = __ldg(up + i);
            i = next < i ? next : -1;   // a parent comes before its child; anything else ends the path
          }
        } else {
#pragma unroll
          for (int e = 0; e < kMaxNodes / 32; ++e)
            see[e] = node >= 32 * e + 31 ? 0xFFFFFFFFu : node >= 32 * e ? (2u << (node - 32 * e)) - 1u : 0u;
        }
      }
      float m_run = -INFINITY, l_run = 0.0f;
      for (int j = seg.j0; j < seg.j1; ++j, ++it) {
        const int sb = it & 1;
        if (!mbar_wait(&s.s_full[sb], (it >> 1) & 1, abort_flag, 0x2501)) { ok = false; break; }
        tc_fence_after();
        if (any_live) {
          float sv[kKeys];
#pragma unroll
          for (int c = 0; c < kKeys / 16; ++c) tmem_ld_x16(tmem + lane_base + TM::s(sb) + c * 16, reinterpret_cast<uint32_t*>(sv) + c * 16);
          tmem_ld_wait();
          reg_fence<kKeys>(reinterpret_cast<uint32_t*>(sv));
          tc_fence_before();
          __syncwarp();
          mbar_arrive_if(&s.s_free[sb], lane == 0);
          if (j == 0) {
#pragma unroll
            for (int c = 0; c < kKeys; ++c)
              if (!((see[c / 32] >> (c % 32)) & 1u)) sv[c] = -INFINITY;
          } else {
            const int cmax = live ? len - (n_blocks - j) * kKeys : 0;
            if (cmax < kKeys) {
#pragma unroll
              for (int c = 0; c < kKeys; ++c)
                if (c >= cmax) sv[c] = -INFINITY;
            }
          }
          float mx;
          {
            float tmp[kKeys];
#pragma unroll
            for (int c = 0; c < kKeys; ++c) tmp[c] = sv[c];
            mx = tree_max3<kKeys>(tmp);
          }
          const float bm = (mx == -INFINITY) ? -INFINITY : mx * sl2;
          const float m_new = fmaxf(m_run, bm);
          const bool need = m_new > m_run + kRescaleLog2;
          const bool later = j > seg.j0;
          const float alpha_n = ex2_approx(m_run - m_new);
          const float alpha = need ? alpha_n : 1.0f;
          l_run = (need && later) ? l_run * alpha_n : l_run;
          m_run = (need || !later) ? m_new : m_run;
          const bool rescale = __any_sync(0xffffffffu, need) && later;
          const float bias = (m_run == -INFINITY) ? 0.0f : -m_run;
          float rs[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          uint32_t pk[kPairs];
#pragma unroll
          for (int c = 0; c < kPairs; ++c) {
            float x0, x1;
            ffma2(x0, x1, sv[2 * c], sv[2 * c + 1], sl2, sl2, bias, bias);
            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
            const int a = (c & 3) * 2;
            fadd2(rs[a], rs[a + 1], rs[a], rs[a + 1], p0, p1);
            pk[c] = pack_half2(p0, p1);
          }
          l_run += ((rs[0] + rs[1]) + (rs[2] + rs[3])) + ((rs[4] + rs[5]) + (rs[6] + rs[7]));
          if (it >= 1 && !mbar_wait(&s.p_free, (it - 1) & 1, abort_flag, 0x2502)) { ok = false; break; }
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < kKeys / 16; ++c) tmem_st_x8(tP + c * 8, pk + c * 8);
          if (rescale) {
            constexpr int kRc = 64;
#pragma unroll
            for (int b0 = 0; b0 < D; b0 += kRc) {
              uint32_t w[kRc];
#pragma unroll
              for (int c = 0; c < kRc / 16; ++c) tmem_ld_x16(tO + b0 + c * 16, w + c * 16);
              tmem_ld_wait();
              reg_fence<kRc>(w);
#pragma unroll
              for (int e = 0; e < kRc; e += 2) {
                float a, b;
                fmul2(a, b, __uint_as_float(w[e]), __uint_as_float(w[e + 1]), alpha, alpha);
                w[e] = __float_as_uint(a);
                w[e + 1] = __float_as_uint(b);
              }
#pragma unroll
              for (int c = 0; c < kRc / 16; ++c) tmem_st_x16(tO + b0 + c * 16, w + c * 16);
            }
          }
          tmem_st_wait();
        } else {
          __syncwarp();
          mbar_arrive_if(&s.s_free[sb], lane == 0);
          // not ahead of the others: an arrival early would stand for one of theirs
          if (it >= 1 && !mbar_wait(&s.p_free, (it - 1) & 1, abort_flag, 0x2503)) { ok = false; break; }
        }
        tc_fence_before();
        __syncwarp();
        mbar_arrive_if(&s.p_full, lane == 0);
      }
      if (ok && !mbar_wait(&s.p_free, (it - 1) & 1, abort_flag, 0x2504)) ok = false;   // the last PV: O is there
      tc_fence_after();
      if (ok) {
        const bool mine = row < p.rows;
        if (seg.whole()) {
          const float inv = l_run > 0.0f ? 1.0f / l_run : 0.0f;
          __half* to = p.o + (bh * p.rows + row) * D;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            uint32_t w[16];
            if (any_live) {
              tmem_ld_x16(tO + c * 16, w);
              tmem_ld_wait();
              reg_fence<16>(w);
            }
            float f[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) f[e] = live ? __uint_as_float(w[column_of(e)]) * inv : 0.0f;
            if (mine) {
#pragma unroll
              for (int e = 0; e < 16; e += 8)
                *reinterpret_cast<uint4*>(to + c * 16 + e) = make_uint4(pack_half2(f[e], f[e + 1]), pack_half2(f[e + 2], f[e + 3]),
                                                                         pack_half2(f[e + 4], f[e + 5]), pack_half2(f[e + 6], f[e + 7]));
            }
          }
          if (mine && p.lse)
            p.lse[bh * p.rows + row] =
                l_run > 0.0f ? (m_run + log2f(l_run)) * 0.69314718055994531f + offset * p.scale : -INFINITY;
        } else {
          const long long slot = 2ll * blockIdx.x + (seg.first ? 0 : 1);
          float4* to = reinterpret_cast<float4*>(p.part_o) + slot * (D / 4) * kRows + r;
          if (any_live) {
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              uint32_t w[16];
              tmem_ld_x16(tO + c * 16, w);
              tmem_ld_wait();
              reg_fence<16>(w);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                to[(c * 4 + e) * kRows] =
                    make_float4(__uint_as_float(w[column_of(4 * e)]), __uint_as_float(w[column_of(4 * e + 1)]),
                                __uint_as_float(w[column_of(4 * e + 2)]), __uint_as_float(w[column_of(4 * e + 3)]));
            }
          }
          p.part_ml[slot * kRows + r] = make_float2(m_run, l_run);
        }
      }
      tc_fence_before();   // O is read before the next segment's first PV, which waits for P
      seg.advance();
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 5) tmem_dealloc(tmem, 512);
}

// Join the partials of the segments that several CTAs shared, and write the rows of sequences without a node. A CTA takes
// 8 channels of a segment's rows, a thread 4 of one row.
template <int D>
__global__ void __launch_bounds__(256) kv4_tree_merge_kernel(const __grid_constant__ Params p) {
  const int per_b = p.Hkv * p.row_tiles;
  const int b = blockIdx.x / per_b, in_b = blockIdx.x % per_b;
  const int weight = p.weight(b);
  const int total = Range::sum(p, p.B) * per_b;
  const int before = Range::sum(p, b) * per_b + in_b * weight;
  griddep_wait();
  const int r = threadIdx.x % kRows, ch = (blockIdx.y * 2 + threadIdx.x / kRows) * 4;
  const int row = in_b % p.row_tiles * kRows + r;
  const long long bh = static_cast<long long>(b) * p.Hkv + in_b / p.row_tiles;
  if (row >= p.rows) return;
  uint2* to = reinterpret_cast<uint2*>(p.o + (bh * p.rows + row) * D + ch);
  const bool dead = weight == 0 || row % p.Sq >= p.count(b);
  if (weight == 0) {
    *to = make_uint2(0u, 0u);
    if (ch == 0 && p.lse) p.lse[bh * p.rows + row] = -INFINITY;
    return;
  }
  const int ctas = min(total, p.ctas);
  const int c0 = Range::cta_of(total, ctas, before + kStart), n = Range::cta_of(total, ctas, before + weight - 1) - c0 + 1;
  if (n == 1) return;   // finished where it was computed
  const int begun = Range::first_of(total, ctas, c0) < before ? 1 : 0;   // c0's first segment was another one
  auto slot = [&](int i) { return 2ll * (c0 + i) + (i == 0 ? begun : 0); };
  float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float mm = -INFINITY, ll = 0.0f;
  if (!dead) {
    for (int i = 0; i < n; ++i) mm = fmaxf(mm, p.part_ml[slot(i) * kRows + r].x);
    for (int i = 0; i < n; ++i) {
      const float2 ml = p.part_ml[slot(i) * kRows + r];
      if (ml.x == -INFINITY) continue;   // a part in which the row sees nothing
      const float f = ex2_approx(ml.x - mm);
      const float4 v = reinterpret_cast<const float4*>(p.part_o)[(slot(i) * (D / 4) + ch / 4) * kRows + r];
      ll = fmaf(f, ml.y, ll);
      x.x = fmaf(f, v.x, x.x), x.y = fmaf(f, v.y, x.y), x.z = fmaf(f, v.z, x.z), x.w = fmaf(f, v.w, x.w);
    }
  }
  const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
  *to = make_uint2(pack_half2(x.x * inv, x.y * inv), pack_half2(x.z * inv, x.w * inv));
  if (ch == 0 && p.lse) {
    float off = 0.0f;
    if (p.shift && !dead) {
      const __half2* q2 = reinterpret_cast<const __half2*>(p.q + (bh * p.rows + row) * D);
      const __half2* m2 = reinterpret_cast<const __half2*>(p.shift + bh * D);
#pragma unroll 16
      for (int c = 0; c < D / 2; ++c) {
        const float2 a = __half22float2(q2[c]), m = __half22float2(m2[c]);
        off = fmaf(a.x, m.x, fmaf(a.y, m.y, off));
      }
    }
    p.lse[bh * p.rows + row] = ll > 0.0f ? (mm + log2f(ll)) * 0.69314718055994531f + off * p.scale : -INFINITY;
  }
}

}  // namespace tree
}  // namespace pasa
