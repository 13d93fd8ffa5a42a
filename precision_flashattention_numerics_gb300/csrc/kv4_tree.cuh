// Attention for drafted tokens over the 4-bit cache of kv4_store.cuh: the query rows of a sequence are the nodes of a tree
// (several guesses of what comes next); each sees the cache's rows, its ancestors and itself. The nodes' own
// keys and values are fp16 and not in the cache yet.
//
// With g heads to a kv head and n nodes a kv head has g n query rows, tens to hundreds, against every cached row: too
// many for kv4_decode_kernel, whose 8 or 16 rows are one side of a mma.sync and which would read and expand the cache once
// for each of them. Here 128 rows are the M side of tcgen05.mma, and a cached row is expanded to fp16 once for all of them.
//
// One CTA works on a segment (sequence, kv head, tile of 128 rows), 128 keys at a time. 28 warps:
//   0-3, 4-7    softmax: two sets, a thread to a row (TMEM lane), that take alternate blocks, so that one's latencies are
//               the other's work (the running maximum goes from set to set through shared memory); and the epilogue
//   8, 9        issue S = Q K'^T and O += P V
//   12-27       expand codes to fp16 tiles in the MMA's swizzled layout: four groups, K' and V of even and of odd blocks, each
//               with the codes of its next block on their way to its registers
// Codes are expanded to s c, which fp16 holds exactly. A word of 8 codes gives the channel order 0, 4, 1, 5, 2, 6, 3, 7 without
// a shuffle; Q is brought to that order when it goes to shared memory, and the epilogue puts O's columns back. P is an
// A operand in TMEM. Scores, maxima, sums and O are fp32, P is rounded to fp16 once (2^-11 of a probability; 2^-24 of
// the row's sum where it is subnormal): what scales it afterwards, when the maximum moves, are powers of two, as maxima are
// whole numbers. (Maxima as they come, with factors in fp16, rounded the probabilities of a row's first blocks up to three times, and
// O apart from the sum. Output errors, relative RMS, of which its own rounding is 2.0e-4: 300 keys 3.31e-4, so 2.90e-4; the largest of
// 28 trees 3.9e-4, so 3.0e-4, or 3.5e-4 with maxima as they come and factors in fp32. Where one key has nearly all of a row's weight its
// probability was 1, which fp16 holds, and is no longer: 61 nodes, uneven, D = 64, 2.12e-4, so 2.86e-4.)
// P overwrites the scores it was made of, 32 columns of S giving 16 of P, so that a row needs 32 scores in registers at a time.
// TMEM holds three S and O: with two S, both sets would wait for PV and QK of their next block before they go on.
// Registers: a launch of 896 threads has 72 each, moved between the roles by setmaxnreg: 2 x 104 + 40 + 4 x 64 <= 7 x 72.
// The roles' loops are kept short (not unrolled over a block): with five roles' code side by side, unrolled loops left the
// warps waiting for instructions most of the time.
//
// Items. A segment is a list of key blocks: first the nodes, then the cache's blocks from its last, partial one
// on.
//
// Work split. The segments' items are numbered in order, a segment's start counting as kStart items, and CTA c takes the
// c-th of equal ranges: uneven lengths keep all SMs equally busy. A segment inside one CTA is finished there, else
// its CTAs leave (O, max, sum) partials that kv4_tree_merge_kernel joins.
//
// The nodes' keys are taken as they are, cached ones lack the shift: the node block's scores lose q . shift in fp32. (Keys
// rounded to fp16 after the shift is taken off moved the LSE of rows that see few keys by up to 4e-5.)
//
// Measured (GPU time per call): 16 nodes x 7 heads x 8 x 32768 keys 85.3 us, of which 79.5 here (issue 56%, tensor pipe 40%: the roles
// wait for one another); 8 nodes on 300 keys 14.4 us; 61 nodes, 6 uneven sequences, D = 64 22.6 us. With 16 rows to a tile on the decode
// kernel the first would take about 250 us.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "attn_fwd.cuh"
#include "kv4_store.cuh"
#include "ptx.cuh"

namespace pasa {
namespace tree {

constexpr int kThreads = 896;
constexpr int kFirstExpand = 12;   // warps
constexpr int kRows = 128;       // of a tile
constexpr int kKeys = 128;       // of a block
constexpr int kMaxNodes = 128;
constexpr int kStages = 3;       // of expanded tiles: 192 KB with D = 128
constexpr int kScores = 3;       // S buffers
constexpr int kCtas = 152;
constexpr int kStart = 4;        // items that the start and end of a segment cost (2: 84.2 us, 4: 81.8, 6: 81.5 for 8 x 32768 keys)
constexpr int kExpandThreads = 128;   // of a tile

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
  int2* parts;                   // [segments]: first partial slot and how many (0: finished where it was computed)
  int B, Hkv, Sq, rows, row_tiles;
  int Sk, cap;
  int ctas;                      // that share all items, or 0: a CTA to a segment
  float scale, scale_log2;

  __device__ __forceinline__ int length(int b) const { return lengths ? min(max(lengths[b], 0), Sk) : Sk; }
  __device__ __forceinline__ int count(int b) const { return counts ? min(max(counts[b], 0), Sq) : Sq; }
};

// Key blocks of a segment, and what it weighs in the shares; 0 without a node.
__device__ __forceinline__ int items_of(int len, int nodes) { return nodes == 0 ? 0 : 1 + (len + kKeys - 1) / kKeys; }
__device__ __forceinline__ int weight_of(int items) { return items == 0 ? 0 : items + kStart; }

// A CTA's range of the items of all segments, and the segments in it, one after another. Made and advanced
// by whole warps.
struct Range {
  const Params& p;
  int len0, nodes0, upto0;   // lane l: of sequence l, and the weights of sequences 0 .. l
  int todo, b, in_b, r0;
  int len, nodes, n_items;   // of the sequence at hand
  int j0, j1;                // items of the segment at hand
  bool first;                // it is the CTA's first

  static __device__ __forceinline__ int scan(int w) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xFFFFFFFFu, w, d);
      if ((threadIdx.x & 31) >= static_cast<unsigned>(d)) w += x;
    }
    return w;
  }
  __device__ __forceinline__ void load(int b0, int& l, int& n, int& upto) const {
    const int i = b0 + (threadIdx.x & 31);
    l = n = 0;
    if (i < p.B) l = p.length(i), n = p.count(i);
    upto = scan(weight_of(items_of(l, n)));
  }
  // The sum of the weights of sequences 0 .. b_end - 1 (per kv head and row tile).
  __device__ __forceinline__ int sum(int b_end) const {
    int total = 0, l, n, upto = upto0;
#pragma unroll 1
    for (int b0 = 0; b0 < b_end; b0 += 32) {
      if (b0 > 0) load(b0, l, n, upto);
      total += __shfl_sync(0xFFFFFFFFu, upto, min(b_end - b0, 32) - 1);
    }
    return total;
  }
  static __device__ __forceinline__ int first_of(int total, int ctas, int c) {
    const int base = total / ctas, more = total - base * ctas;
    return c * base + min(c, more);
  }
  __device__ __forceinline__ explicit Range(const Params& params) : p(params), todo(0), first(true) {
    if (p.ctas > 0) load(0, len0, nodes0, upto0);
  }
  __device__ __forceinline__ int per_b() const { return p.Hkv * p.row_tiles; }
  // The range of a CTA: this one's in the attention kernel.
  __device__ __forceinline__ void start(int cta) {
    if (p.ctas == 0) {
      b = cta / per_b();
      in_b = cta % per_b();
      len = p.length(b);
      nodes = p.count(b);
      n_items = items_of(len, nodes);
      todo = weight_of(n_items);
      r0 = -kStart;
      return;
    }
    const int total = sum(p.B) * per_b(), ctas = min(total, p.ctas);
    if (cta >= ctas) return;
    int place = first_of(total, ctas, cta);
    todo = first_of(total, ctas, cta + 1) - place;
    int l = len0, n = nodes0, upto = upto0;
#pragma unroll 1
    for (int b0 = 0;; b0 += 32) {   // place is less than the sum
      if (b0 > 0) load(b0, l, n, upto);
      const uint32_t past = __ballot_sync(0xFFFFFFFFu, upto * per_b() > place);
      if (past != 0) {
        const int lane = __ffs(past) - 1;
        b = b0 + lane;
        len = __shfl_sync(0xFFFFFFFFu, l, lane);
        nodes = __shfl_sync(0xFFFFFFFFu, n, lane);
        n_items = items_of(len, nodes);
        place -= (__shfl_sync(0xFFFFFFFFu, upto, lane) - weight_of(n_items)) * per_b();
        break;
      }
      place -= __shfl_sync(0xFFFFFFFFu, upto, 31) * per_b();
    }
    in_b = place / weight_of(n_items);
    r0 = place - in_b * weight_of(n_items) - kStart;
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
    if (todo > 0 && ++in_b == per_b()) {
      in_b = 0;
      do {
        ++b;   // read again, from L1: registers are short
        len = p.length(b);
        nodes = p.count(b);
        n_items = items_of(len, nodes);
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
  alignas(1024) uint8_t k[kStages][kTile];
  alignas(1024) uint8_t v[kStages][kTile];
  alignas(1024) uint8_t q[kTile];
  uint64_t k_full[kStages], k_empty[kStages];     // expanded (4 warps); QK done
  uint64_t v_full[kStages], v_empty[kStages];
  uint64_t q_full;                                // Q of a segment is there (8 warps)
  uint64_t m_full[4][2];                          // [rows 32 q ..][set]: the set has published m of its block
  uint64_t s_full[kScores], p_full[kScores], p_free[kScores];   // QK done; P written (4 warps); PV done, S may be rewritten
  uint64_t drain[2];
  float m[2][kRows];         // [set]: the maximum that a row's last block was taken with
  uint32_t tmem_base;
  int abort_flag;
};

template <int D>
struct Tmem {
  __host__ __device__ static constexpr int s(int b) { return b * kKeys; }
  static constexpr int o = kScores * kKeys;
  __host__ __device__ static constexpr int sums(int set) { return set * 16; }   // of a segment, from set to set, when S is free
  static_assert(o + D <= 512, "TMEM budget");
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

// 8 codes times the scale, exactly, in the order above: one fused multiply-add for two of them. A nibble moved to bits 6 .. 9 of
// the mantissa of 16 is 16 + n, so (16 + n) s - 24 s = (n - 8) s, which fp16 holds, as it does 24 s (s has 8 bits), up to
// s = 2729. kv4_expand, for any s, takes two such operations, and those bound these loops.
__device__ __forceinline__ uint4 expand8(uint32_t w, __half2 s2, __half2 minus24s) {
  const uint32_t nibble = 0x03C003C0u, sixteen = 0x4C004C00u;
  const __half2 a = __hfma2(bits_h2(((w << 6) & nibble) | sixteen), s2, minus24s);
  const __half2 b = __hfma2(bits_h2(((w << 2) & nibble) | sixteen), s2, minus24s);
  const __half2 c = __hfma2(bits_h2(((w >> 2) & nibble) | sixteen), s2, minus24s);
  const __half2 d = __hfma2(bits_h2(((w >> 6) & nibble) | sixteen), s2, minus24s);
  return make_uint4(h2_bits(a), h2_bits(b), h2_bits(c), h2_bits(d));
}
// 16 bytes of codes and their scale, or zeros where `there` is false (nothing is read then). In one piece: a branch around the
// loads would end in moves of what they bring, which wait for it.
__device__ __forceinline__ void load_chunk(uint4& x, unsigned short& scale, const uint8_t* codes, const __half* scales, bool there) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %7, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\tmov.b16 %4, 0;\n\t"
      "@p ld.global.cs.v4.b32 {%0, %1, %2, %3}, [%5];\n\t"
      "@p ld.global.b16 %4, [%6];\n\t}"
      : "=&r"(x.x), "=&r"(x.y), "=&r"(x.z), "=&r"(x.w), "=&h"(scale)
      : "l"(codes), "l"(scales), "r"(there ? 1u : 0u)
      : "memory");
}
// 16 bytes, or zeros where `there` is false, in one piece for the same reason.
__device__ __forceinline__ uint4 load16_if(const void* from, bool there) {
  uint4 x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %5, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@p ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(x.x), "=&r"(x.y), "=&r"(x.z), "=&r"(x.w)
      : "l"(from), "r"(there ? 1u : 0u)
      : "memory");
  return x;
}
// A chunk, 32 channels of a row, to its four places in a tile: `at` and its neighbours by the units' numbers.
__device__ __forceinline__ void put_chunk(uint32_t at, uint4 codes, unsigned short scale_bits) {
  const __half scale = __ushort_as_half(scale_bits);
  const __half2 s2 = __half2half2(scale);
  auto store = [&](uint32_t to, uint4 y) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w) : "memory");
  };
  if (__half2float(scale) <= 2729.0f) {
    const __half2 m = __hmul2(s2, __float2half2_rn(-24.0f));
    store(at, expand8(codes.x, s2, m));
    store(at ^ 16, expand8(codes.y, s2, m));
    store(at ^ 32, expand8(codes.z, s2, m));
    store(at ^ 48, expand8(codes.w, s2, m));
  } else {
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      __half2 h[4];
      kv4_expand(codes.x, s2, h);
      store(at ^ (16 * i), make_uint4(h2_bits(h[0]), h2_bits(h[1]), h2_bits(h[2]), h2_bits(h[3])));
      codes = make_uint4(codes.y, codes.z, codes.w, codes.x);
    }
  }
}

// 2^d of a whole number d <= 0 or -inf, exactly; 0 below the least normal number.
__device__ __forceinline__ float power_of_two(float d) { return d < -126.0f ? 0.0f : __int_as_float((static_cast<int>(d) + 127) << 23); }

// The first n of 32 bits.
__device__ __forceinline__ uint32_t first_bits(int n) { return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u; }
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
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s.k_full[i], 4);
      mbar_init(&s.k_empty[i], 1);
      mbar_init(&s.v_full[i], 4);
      mbar_init(&s.v_empty[i], 1);
    }
    for (int i = 0; i < kScores; ++i) {
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.p_free[i], 1);
      mbar_init(&s.p_full[i], 4);
    }
    mbar_init(&s.q_full, 8);
    for (int i = 0; i < 4; ++i) mbar_init(&s.m_full[i][0], 1), mbar_init(&s.m_full[i][1], 1);
    mbar_init(&s.drain[0], 1);
    mbar_init(&s.drain[1], 1);
    s.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(&s.tmem_base, 512);
    tmem_relinquish();
  }
  Range seg(p);   // its loads are on their way while the barriers are made
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  volatile int* abort_flag = &s.abort_flag;
  seg.start(blockIdx.x);

  if (warp >= kFirstExpand) {
    // ------------------------------------------------------------------ codes to fp16
    // Four warps to a group: K' and V tiles of even items, then of odd ones. One warp of the four looks at the barrier, the
    // others wait for it at a named one, which takes no issue slots.
    regs_down<64>();
    const int group = (warp - kFirstExpand) / 4, mine = group >> 1;
    const bool values = group & 1;
    const int t = (tid - kFirstExpand * 32) % kExpandThreads;
    constexpr int kGroups = D / 32;                              // 16-byte chunks of a row of codes
    constexpr int kPer = kKeys * kGroups / kExpandThreads;       // of a tile, for a thread
    constexpr int kRowStep = kExpandThreads / kGroups;
    // of a thread's chunks: group w of row row_t, kRowStep rows apart. 8 neighbouring lanes have 4 rows of one 64-channel
    // column, and their units of 16 bytes fall into 8 different bank groups.
    const int w = (t & 1) + (D == 128 ? (t >> 3 & 1) * 2 : 0), row_t = D == 128 ? (t >> 1 & 3) + (t >> 4) * 4 : t >> 1;
    const uint32_t place = smem_u32(values ? s.v[0] : s.k[0]) + (w >> 1) * S::kChunk + row_t * 128 + ((((w & 1) * 4) ^ (row_t & 7)) * 16);
    uint64_t *full = values ? s.v_full : s.k_full, *empty = values ? s.v_empty : s.k_empty;
    int it = 0;
    bool ok = true;
    while (ok && seg.next()) {
      const int it0 = it, skip = (it & 1) != mine ? 1 : 0;
      // a thread's first row of the next item, which is two blocks further to the front of the cache, and how many rows from there
      // on the sequence has: what lies past its last row is 0 and not read
      const long long row = seg.head() * p.cap + static_cast<long long>(seg.n_items - 1 - seg.j0 - skip) * kKeys + row_t;
      const uint8_t* codes = (values ? p.v4 : p.k4) + row * (D / 2) + w * 16;
      const __half* scales = (values ? p.vscale : p.kscale) + row * kGroups + w;
      int left = seg.j0 + skip > 0 && seg.j0 + skip < seg.j1 ? seg.len - (seg.n_items - 1 - seg.j0 - skip) * kKeys - row_t : 0;
      uint4 x[kPer];
      unsigned short scale[kPer];
      auto fetch = [&](int i) {
        load_chunk(x[i], scale[i], codes + i * (kRowStep * D / 2), scales + i * (kRowStep * kGroups), i * kRowStep < left);
      };
#pragma unroll
      for (int i = 0; i < kPer; ++i) fetch(i);
#pragma unroll 1
      for (int j = seg.j0 + skip; j < seg.j1; j += 2) {
        it = it0 + j - seg.j0;
        const int stage = it % kStages;
        uint8_t* tile = (values ? s.v : s.k)[stage];
        bool go = true;
        if (warp % 4 == 0 && it >= kStages) go = mbar_wait(&empty[stage], (it / kStages - 1) & 1, abort_flag, 0x2101);
        if (!named_bar_and(2 + group, kExpandThreads, go)) { ok = false; break; }
        codes -= 2 * kKeys * (D / 2);
        scales -= 2 * kKeys * kGroups;
        left = j + 2 < seg.j1 ? kKeys : 0;
        if (j > 0) {
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            put_chunk(place + stage * S::kTile + i * (kRowStep * 128), x[i], scale[i]);
            fetch(i);
          }
        } else {
          // the nodes: K or V in fp16, rows past the last node 0
#pragma unroll
          for (int i = 0; i < kPer; ++i) fetch(i);
          const long long bh = seg.head();
          const __half* from = (values ? p.v : p.k) + bh * p.Sq * D;
          constexpr int kUnits = D / 8, kStep = kExpandThreads / kUnits;
          const int u = t % kUnits;
#pragma unroll 1
          for (int r = t / kUnits; r < kKeys; r += 2 * kStep) {
            uint4 y[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) y[i] = load16_if(from + (r + i * kStep) * D + u * 8, r + i * kStep < seg.nodes);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int row = r + i * kStep;
              *reinterpret_cast<uint4*>(tile + (u / 8) * S::kChunk + row * 128 + (((u % 8) ^ (row & 7)) * 16)) = code_order(y[i]);
            }
          }
        }
        fence_proxy_async_smem();   // the MMA reads the tile through the async proxy
        __syncwarp();
        mbar_arrive_if(&full[stage], lane == 0);
      }
      it = it0 + seg.j1 - seg.j0;
      seg.advance();
    }
  } else if (warp >= 8) {
    regs_down<40>();
    if (warp == 8) {
      // ---------------------------------------------------------------- S = Q K'^T
      constexpr uint32_t id_s = idesc_f16(kRows, kKeys, true, false);
      constexpr uint32_t hi = sdesc_hi_sw128(1024);
      const uint32_t k_lo = sdesc_lo(smem_u32(s.k[0]), 16), q_lo = sdesc_lo(smem_u32(s.q), 16);
      int it = 0, nth = 0;
      bool ok = true;
      while (ok && seg.next()) {
        if (!mbar_wait(&s.q_full, nth & 1, abort_flag, 0x2301)) break;
#pragma unroll 1
        for (int j = seg.j0; j < seg.j1; ++j, ++it) {
          const int st = it % kStages, sb = it % kScores;
          if (!mbar_wait(&s.k_full[st], (it / kStages) & 1, abort_flag, 0x2302)) { ok = false; break; }
          if (it >= kScores && !mbar_wait(&s.p_free[sb], (it / kScores - 1) & 1, abort_flag, 0x2303)) { ok = false; break; }
          tc_fence_after();
          if (lane == 0) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = ((kk / 4) * S::kChunk + (kk % 4) * 32) >> 4;
              mma_ss_w(tmem + TM::s(sb), q_lo + off, hi, k_lo + (st * S::kTile >> 4) + off, hi, id_s, kk > 0 ? 1u : 0u);
            }
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
    } else if (warp == 9) {
      // ---------------------------------------------------------------- O += P V
      constexpr uint32_t id_o = idesc_f16(kRows, D, true, true);
      constexpr uint32_t hi = sdesc_hi_sw128(1024);
      const uint32_t v_lo = sdesc_lo(smem_u32(s.v[0]), S::kChunk);
      int it = 0;
      bool ok = true;
      while (ok && seg.next()) {
#pragma unroll 1
        for (int j = seg.j0; j < seg.j1; ++j, ++it) {
          const int st = it % kStages, sb = it % kScores;
          if (!mbar_wait(&s.v_full[st], (it / kStages) & 1, abort_flag, 0x2401)) { ok = false; break; }
          if (!mbar_wait(&s.p_full[sb], (it / kScores) & 1, abort_flag, 0x2402)) { ok = false; break; }
          tc_fence_after();
          if (lane == 0) {
            const uint32_t more = j > seg.j0 ? 1u : 0u;
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
              mma_ts_w(tmem + TM::o, tmem + TM::s(sb) + kk * 8, v_lo + ((st * S::kTile + kk * 2048) >> 4), hi, id_o, kk > 0 ? 1u : more);
            mma_commit(&s.p_free[sb]);
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
    // Warps q and q + 4 have the rows 32 q ..: of Q's and O's channels half each, and the blocks in turn. All waits are mbarriers'
    // or end in one barrier of the eight warps for each segment, at which they also agree to stop.
    regs_up<104>();
    const int quad = warp & 3, set = warp >> 2;
    const int r = quad * 32 + lane;
    const uint32_t tmem_q = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    constexpr int kCols = D / 2;
    const uint32_t tO = tmem_q + TM::o;
    const float sl2 = p.scale_log2;
    if (p.ctas == 0 && seg.todo == 0) {   // a sequence without a node
      const int row = seg.row0() + r;
      if (row < p.rows) {
        __half* to = p.o + (seg.head() * p.rows + row) * D + set * kCols;
#pragma unroll 1
        for (int c = 0; c < kCols; c += 8) *reinterpret_cast<uint4*>(to + c) = make_uint4(0u, 0u, 0u, 0u);
        if (set == 0 && p.lse) p.lse[seg.head() * p.rows + row] = -INFINITY;
      }
    }
    int it = 0;
    bool ok = true;
    while (ok && seg.next()) {
      const long long bh = seg.head();
      const int row = seg.row0() + r;
      const int n_blocks = seg.n_items - 1;
      const int node = row % p.Sq;
      const bool live = row < p.rows && node < seg.nodes;
      const bool any_live = __any_sync(0xFFFFFFFFu, live);   // a warp without one only keeps the barriers going
      const int* up = p.parents + static_cast<long long>(seg.b) * p.Sq;
      if (p.parents && seg.j0 == 0 && any_live)   // into L1, ahead of the walk
        asm volatile("prefetch.global.L1 [%0];" ::"l"(up + min(lane * 4, p.Sq - 1)));
      // Q to shared memory; the QKs of the segment before are done, as both sets have come to its end. And q . shift, which cached
      // keys lack and the nodes' have: half of the channels each, exchanged through S's columns, which are free until Q is there.
      float offset = 0.0f;
      const bool shifted = p.shift != nullptr && (seg.j0 == 0 || (p.lse != nullptr && seg.whole()));
      if (any_live) {
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (bh * p.rows + row) * D) + set * (D / 16);
        uint4 x[D / 16];
#pragma unroll
        for (int i = 0; i < D / 16; ++i) x[i] = load16_if(src + i, live);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const int u = set * (D / 16) + i;
          *reinterpret_cast<uint4*>(s.q + (u / 8) * S::kChunk + r * 128 + (((u % 8) ^ (r & 7)) * 16)) = code_order(x[i]);
        }
        fence_proxy_async_smem();
        if (shifted) {
          const uint4* sh = reinterpret_cast<const uint4*>(p.shift + bh * D) + set * (D / 16);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const uint4 y = __ldg(sh + i);
            const uint32_t xa[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, ya[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 a = __half22float2(bits_h2(xa[e])), m = __half22float2(bits_h2(ya[e]));
              offset = fmaf(a.x, m.x, fmaf(a.y, m.y, offset));
            }
          }
          tmem_st_x1(tmem_q + TM::sums(set), __float_as_uint(offset));
          tmem_st_wait();
        }
      }
      if (shifted) {
        tc_fence_before();
        named_bar_sync(1, 256);
        tc_fence_after();
        if (any_live) {
          uint32_t other;
          tmem_ld_x1(tmem_q + TM::sums(set ^ 1), other);
          tmem_ld_wait();
          reg_fence<1>(&other);
          offset += __uint_as_float(other);
        }
        tc_fence_before();
      }
      __syncwarp();
      mbar_arrive_if(&s.q_full, lane == 0);
      // the nodes that this row's node sees
      uint32_t see[kMaxNodes / 32] = {};
      if (live && seg.j0 == 0 && (it & 1) == set) {
        if (p.parents) {
#pragma unroll 1
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
      float m_w = -INFINITY, l_w = 0.0f;   // this set's sum, and the maximum it is scaled to
      int j = seg.j0 + ((it & 1) != set ? 1 : 0);
      const int it0 = it;
      for (it += j - seg.j0; j < seg.j1; j += 2, it += 2) {
        const int sb = it % kScores;
        const uint32_t tS = tmem_q + TM::s(sb);
        if (!mbar_wait(&s.s_full[sb], (it / kScores) & 1, abort_flag, 0x2501)) { ok = false; break; }
        tc_fence_after();
        if (any_live) {
          // 32 keys at a time: exponentials against the maximum at hand, which moves when a score passes it by more than 8
          // (log2 units); what was taken against the one before is then scaled. Maxima are whole numbers (rounded down, so that a
          // row's largest probability is 1 at least, and its sum) and factors so powers of two: P, the sums and O are scaled
          // without a rounding, but for probabilities that become subnormal in fp16. Rows without a node have zeros for Q, and
          // nothing of theirs is kept: but for the nodes, all rows have the same keys.
          const int keys = j == 0 ? 0 : seg.len - (n_blocks - j) * kKeys;
          const bool later = j > seg.j0;
          const float less = j == 0 ? offset : 0.0f;   // the nodes' keys are not shifted
          float m_cur = m_w, l = 0.0f;
          auto scale_p = [&](int columns, float f) {   // 16 columns of P at a time
            f = fmaxf(f, 0x1p-48f);   // which leaves nothing of a probability in fp16
#pragma unroll 1
            do {   // once, but where f is below fp16's least number, 2^-24
              tmem_st_wait();   // they may just have been stored, and a load does not wait for stores by itself
              const float f16 = fmaxf(f, 0x1p-24f);
              const uint32_t f2 = pack_half2(f16, f16);
#pragma unroll 1
              for (int c = 0; c < columns; c += 16) {
                uint32_t w[16];
                tmem_ld_x16(tS + c, w);
                tmem_ld_wait();
                reg_fence<16>(w);
#pragma unroll
                for (int e = 0; e < 16; ++e) w[e] = hmul2(w[e], f2);
                tmem_st_x16(tS + c, w);
              }
              f = fminf(f * 0x1p24f, 1.0f);
            } while (__any_sync(0xffffffffu, f < 1.0f));
            tmem_st_wait();
          };
#pragma unroll 1
          for (int c = 0; c < kKeys / 32; ++c) {
            float sv[32];
            tmem_ld_x16(tS + c * 32, reinterpret_cast<uint32_t*>(sv));
            tmem_ld_x16(tS + c * 32 + 16, reinterpret_cast<uint32_t*>(sv) + 16);
            tmem_ld_wait();
            reg_fence<32>(reinterpret_cast<uint32_t*>(sv));
            if (keys < kKeys) {
              const uint32_t bits = j > 0 ? first_bits(keys - 32 * c) : c == 0 ? see[0] : c == 1 ? see[1] : c == 2 ? see[2] : see[3];
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((bits >> e) & 1u)) sv[e] = -INFINITY;
            }
            float top[11];
#pragma unroll
            for (int e = 0; e < 10; ++e) top[e] = fmax3(sv[3 * e], sv[3 * e + 1], sv[3 * e + 2]);
            top[10] = fmaxf(sv[30], sv[31]);
            const float most = (tree_max3<11>(top) - less) * sl2;
            const bool need = most > m_cur + kRescaleLog2;
            if (__any_sync(0xffffffffu, need)) {
              const float m_new = need ? floorf(most) : m_cur;
              const float f = need ? power_of_two(m_cur - m_new) : 1.0f;
              m_cur = m_new;
              l *= f;
              if (c > 0) scale_p(c * 16, f);
            }
            const float bias = (m_cur == -INFINITY) ? 0.0f : -less * sl2 - m_cur;
            float rs[4] = {0.f, 0.f, 0.f, 0.f};
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float x0, x1;
              ffma2(x0, x1, sv[2 * e], sv[2 * e + 1], sl2, sl2, bias, bias);
              const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
              fadd2(rs[2 * (e & 1)], rs[2 * (e & 1) + 1], rs[2 * (e & 1)], rs[2 * (e & 1) + 1], p0, p1);
              pk[e] = pack_half2(p0, p1);
            }
            tmem_st_x16(tS + c * 16, pk);
            l += (rs[0] + rs[1]) + (rs[2] + rs[3]);
          }
          tmem_st_wait();
          // the other set's block in between may have moved the maximum too: O is scaled to m_prev
          float m_prev = m_cur;
          if (later) {
            if (!mbar_wait(&s.m_full[quad][set ^ 1], ((it - 1) >> 1) & 1, abort_flag, 0x2505)) { ok = false; break; }
            m_prev = s.m[set ^ 1][r];
          }
          const float m_end = fmaxf(m_prev, m_cur);
          s.m[set][r] = m_end;
          __syncwarp();
          mbar_arrive_if(&s.m_full[quad][set], lane == 0);
          if (__any_sync(0xffffffffu, m_end > m_cur)) {
            const float f = m_end > m_cur ? power_of_two(m_cur - m_end) : 1.0f;
            l *= f;
            scale_p(kKeys / 2, f);
          }
          if (m_w != m_end) l_w *= power_of_two(m_w - m_end);   // 0 while this set has no block yet
          l_w += l;
          m_w = m_end;
          if (__any_sync(0xffffffffu, later && m_end > m_prev)) {
            const float alpha = m_end > m_prev ? power_of_two(m_prev - m_end) : 1.0f;
            if (!mbar_wait(&s.p_free[(it - 1) % kScores], ((it - 1) / kScores) & 1, abort_flag, 0x2502)) { ok = false; break; }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t w[16];
              tmem_ld_x16(tO + c, w);
              tmem_ld_wait();
              reg_fence<16>(w);
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * alpha);
              tmem_st_x16(tO + c, w);
            }
            tmem_st_wait();
          }
        } else {
          mbar_arrive_if(&s.m_full[quad][set], lane == 0);   // nobody waits for it, but its phases count items
        }
        tc_fence_before();
        __syncwarp();
        mbar_arrive_if(&s.p_full[sb], lane == 0);
      }
      it = it0 + seg.j1 - seg.j0;
      // the last PV: O is there
      if (ok) ok = mbar_wait(&s.p_free[(it - 1) % kScores], ((it - 1) / kScores) & 1, abort_flag, 0x2504);
      tc_fence_after();
      // Only of the set that had the last item is this sure (the other may see the phase of two PVs before): so after the
      // barrier for both. Then the sets exchange their sums through S's columns.
      ok = named_bar_and(1, 256, ok);
      uint32_t w16[16] = {__float_as_uint(l_w), __float_as_uint(m_w)};
      if (ok) {
        tmem_st_x16(tmem_q + TM::sums(set), w16);
        tmem_st_wait();
      }
      tc_fence_before();
      named_bar_sync(1, 256);
      tc_fence_after();
      if (ok) {
        tmem_ld_x16(tmem_q + TM::sums(set ^ 1), w16);
        tmem_ld_wait();
        reg_fence<16>(w16);
        const float2 other = make_float2(__uint_as_float(w16[0]), __uint_as_float(w16[1]));
        float m_run = fmaxf(m_w, other.y);   // what O is scaled to: the last block's
        // without a maximum both sums are 0, or NaN for a NaN query
        float l_run = m_run == -INFINITY ? l_w + other.x : l_w * ex2_approx(m_w - m_run) + other.x * ex2_approx(other.y - m_run);
        if (!live) m_run = -INFINITY, l_run = 0.0f;
        const bool mine = row < p.rows;
        const uint32_t tMine = tO + set * kCols;
        if (seg.whole()) {
          const float inv = l_run == 0.0f ? 0.0f : 1.0f / l_run;
          __half* to = p.o + (bh * p.rows + row) * D + set * kCols;
#pragma unroll
          for (int c = 0; c < kCols / 16; ++c) {
            uint32_t w[16];
            if (any_live) {
              tmem_ld_x16(tMine + c * 16, w);
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
          if (tid == 0 && p.ctas > 0) p.parts[seg.b * seg.per_b() + seg.in_b] = make_int2(0, 0);
          if (mine && set == 0 && p.lse)
            p.lse[bh * p.rows + row] =
                l_run == 0.0f ? -INFINITY : (m_run + log2f(l_run)) * 0.69314718055994531f + offset * p.scale;
        } else {
          const long long slot = 2ll * blockIdx.x + (seg.first ? 0 : 1);
          float4* to = reinterpret_cast<float4*>(p.part_o) + (slot * (D / 4) + set * (kCols / 4)) * kRows + r;
          if (any_live) {
#pragma unroll
            for (int c = 0; c < kCols / 16; ++c) {
              uint32_t w[16];
              tmem_ld_x16(tMine + c * 16, w);
              tmem_ld_wait();
              reg_fence<16>(w);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                to[(c * 4 + e) * kRows] =
                    make_float4(__uint_as_float(w[column_of(4 * e)]), __uint_as_float(w[column_of(4 * e + 1)]),
                                __uint_as_float(w[column_of(4 * e + 2)]), __uint_as_float(w[column_of(4 * e + 3)]));
            }
          }
          if (set == 0) p.part_ml[slot * kRows + r] = make_float2(m_run, l_run);
          // the first part's CTA says where the parts begin, the last one's where they end
          if (tid == 0 && seg.j0 == 0) p.parts[seg.b * seg.per_b() + seg.in_b].x = static_cast<int>(slot);
          if (tid == 0 && seg.j1 == seg.n_items) p.parts[seg.b * seg.per_b() + seg.in_b].y = static_cast<int>(blockIdx.x) + 1;
        }
      }
      // O is read before the next segment's first PV, which waits for P, and the sums before they are written again
      tc_fence_before();
      named_bar_sync(1, 256);
      seg.advance();
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

// Join the partials of the segments that several CTAs shared. A CTA takes 8 channels of a segment's rows, a thread 4 of
// one row. With no more segments than CTAs that share them, blockIdx.x is a segment. With more, most of which end where they
// began, it is a CTA c of the kernel before, and the segment the one in which the range of c ends, if it began there (512
// segments on 1024 keys: with a CTA for each 81.6 us in all, so 71.8; 2048 of them: 320, 264). The blocks behind those write the rows of sequences without a node.
template <int D, bool BY_SEGMENT>
__global__ void __launch_bounds__(256) kv4_tree_merge_kernel(const __grid_constant__ Params p) {
  const int per_b = p.Hkv * p.row_tiles, places = BY_SEGMENT ? p.B * per_b : p.ctas - 1;
  if (static_cast<int>(blockIdx.x) >= places) {
    griddep_wait();
    const long long rows = static_cast<long long>(p.Hkv) * p.rows;   // of a sequence
    const long long first = static_cast<long long>(blockIdx.y) * 256 + threadIdx.x, step = gridDim.y * 256ll;
    for (int b = blockIdx.x - places; b < p.B; b += gridDim.x - places) {
      if (p.count(b) != 0) continue;
      uint4* to = reinterpret_cast<uint4*>(p.o + b * rows * D);
      for (long long i = first; i < rows * (D / 8); i += step) to[i] = make_uint4(0u, 0u, 0u, 0u);
      for (long long i = first; p.lse && i < rows; i += step) p.lse[b * rows + i] = -INFINITY;
    }
    return;
  }
  int b, in_b, nodes;
  if constexpr (BY_SEGMENT) {
    b = blockIdx.x / per_b, in_b = blockIdx.x % per_b;
    nodes = p.count(b);
  } else {
    Range next(p);
    next.start(blockIdx.x + 1);
    if (next.todo <= 0 || next.r0 <= 0) {   // no CTA behind this one, or it begins with a segment
      griddep_wait();
      return;
    }
    b = next.b, in_b = next.in_b, nodes = next.nodes;
  }
  const int r = threadIdx.x % kRows, ch = (blockIdx.y * 2 + threadIdx.x / kRows) * 4;
  const int row = in_b % p.row_tiles * kRows + r;
  const long long bh = static_cast<long long>(b) * p.Hkv + in_b / p.row_tiles;
  griddep_wait();
  if (row >= p.rows || nodes == 0) return;
  const int2 parts = __ldcg(p.parts + static_cast<long long>(b) * per_b + in_b);
  if (parts.y == 0) return;   // finished where it was computed
  // slots: the first part's, and the first of each of the following CTAs (kept in range where a call has failed and left no numbers)
  const int slot0 = min(static_cast<unsigned>(parts.x), 2u * kCtas - 1), cta = slot0 >> 1, n = min(parts.y, kCtas) - cta;
  if (!BY_SEGMENT && cta != static_cast<int>(blockIdx.x)) return;   // it began before
  float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float mm = -INFINITY, ll = 0.0f;
  if (row % p.Sq < nodes) {
    constexpr int kAtOnce = 8;
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += kAtOnce) {
      float2 ml[kAtOnce];
      float4 v[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const long long slot = i0 + i == 0 ? slot0 : 2ll * (cta + i0 + i);
        ml[i] = make_float2(-INFINITY, 0.0f);
        v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (i0 + i < n) {
          ml[i] = __ldcg(p.part_ml + slot * kRows + r);
          v[i] = __ldcg(reinterpret_cast<const float4*>(p.part_o) + (slot * (D / 4) + ch / 4) * kRows + r);
        }
      }
      float top = mm;
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) top = fmaxf(top, ml[i].x);
      if (top == -INFINITY) {   // parts in which the row sees nothing, or of a NaN query, whose sums are NaN
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) ll += ml[i].y;
        continue;
      }
      const float f0 = ex2_approx(mm - top);
      ll *= f0, x.x *= f0, x.y *= f0, x.z *= f0, x.w *= f0;
      mm = top;
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const float f = ex2_approx(ml[i].x - mm);
        ll = fmaf(f, ml[i].y, ll);
        x.x = fmaf(f, v[i].x, x.x), x.y = fmaf(f, v[i].y, x.y), x.z = fmaf(f, v[i].z, x.z), x.w = fmaf(f, v[i].w, x.w);
      }
    }
  }
  const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
  *reinterpret_cast<uint2*>(p.o + (bh * p.rows + row) * D + ch) = make_uint2(pack_half2(x.x * inv, x.y * inv), pack_half2(x.z * inv, x.w * inv));
  if (ch == 0 && p.lse) {
    float off = 0.0f;
    if (p.shift && ll != 0.0f) {
      const uint4* q4 = reinterpret_cast<const uint4*>(p.q + (bh * p.rows + row) * D);
      const uint4* m4 = reinterpret_cast<const uint4*>(p.shift + bh * D);
#pragma unroll 4
      for (int c = 0; c < D / 8; ++c) {
        const uint4 qa = __ldg(q4 + c), ma = __ldg(m4 + c);
        const uint32_t qw[4] = {qa.x, qa.y, qa.z, qa.w}, mw[4] = {ma.x, ma.y, ma.z, ma.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 a = __half22float2(bits_h2(qw[e])), m = __half22float2(bits_h2(mw[e]));
          off = fmaf(a.x, m.x, fmaf(a.y, m.y, off));
        }
      }
    }
    p.lse[bh * p.rows + row] = ll == 0.0f ? -INFINITY : (mm + log2f(ll)) * 0.69314718055994531f + off * p.scale;
  }
}

}  // namespace tree
}  // namespace pasa
