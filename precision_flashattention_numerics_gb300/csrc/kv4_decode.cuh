// Decode attention on the 4-bit cache of kv4_store.cuh: a few query rows per head against
// cached keys and values, O = softmax(scale * q K'^T) V, and the attention weight each cached
// row gets. One shift per kv head and channel is the same for every key of a row, so
// q . shift cancels in the softmax and only enters the log-sum-exp.
//
// kv4_decode_kernel. HBM-bound for up to 8 rows: 9 D / 8 bytes per cached row of K and V against
// 4 rows D flops. A warp takes 32 keys at a time: codes by cp.async to its own two stages of shared
// memory, from there by ldmatrix into the registers of mma.sync m16n8k16 (fp16 in, fp32 out):
//   8 rows:  S^T[key][row] = K' Q^T (A = K', 16 keys), O^T[channel][row] += V^T P^T (A = V^T);
//   16 rows: S[row][key] = Q K'^T (A = Q), O[row][channel] += P V (A = P).
// The rows' side is 8 or 16 wide, so that little of an MMA is padding. tcgen05 takes its operands
// from shared or tensor memory, where the expanded codes, four times the bytes that HBM delivers,
// would have to be written and read again; mma.sync takes them from the registers they
// are expanded in.
//   - Keys are not expanded at all: a code masked out of its byte is a subnormal fp16 number, and
//     what it lacks of its value (the -8, the scale) is a constant of the accumulator and one fp32
//     product per score and group of 32 channels (Kv4Query).
//   - Values are expanded to s c, exact in fp16 as s has 8 significant bits. ldmatrix.trans gives a
//     lane 4 channels of two neighbouring keys, the pair that the MMA wants in a register.
//   - P is rounded to fp16 (relative 2^-11, as in the other decode kernels). Scores, maxima, sums and
//     O are fp32.
//
// Work split. A segment is a (sequence, kv head, tile of 8 or 16 rows). Either a cluster of CTAs takes
// a segment, warps interleaved, and joins through distributed shared memory: one launch, no workspace.
// Or (STREAM_K) the segments' rounds are numbered in order and CTA c takes the c-th of gridDim.x equal
// ranges, so that uneven lengths keep all SMs equally busy; a segment inside one CTA is finished
// there, else its CTAs leave (O, max, sum) partials that kv4_merge_kernel joins. Which one is
// chosen on the host by the sizes.
//
// Measured, GPU time of a call in a replayed graph at 2070 MHz: 8 sequences x 4 kv heads x 32768 keys, D = 128, 7 rows:
// 34.7 us for 151 MB, 0.65 of the copy rate; x 131072 keys 109.4 us, 0.83. The two differ by 239 cycles for each 32 keys of
// an SM, where HBM alone takes 217 (0.91 of the copy rate) and a warp's 540 or so instructions take 135 of the SM's
// issue slots. The other 9.7 us do not grow with the keys: 1.7 that any kernel takes in a graph, 3.2 for lengths, shares, the
// first keys and the join (a call of this form with 32 keys in each sequence takes 4.9 without its merge), 2.8 for the
// merge kernel (1.0 where it has nothing to join), and about 2 for the first burst of codes of all CTAs at once and an uneven
// end. Expanding keys like values took 650 instructions (39.5 us); a third CTA per SM needs 80 registers and spills
// (44 us). With D = 128 the kernels kept spill a little too, bytes stored by a thread: shared out 24 (8 rows) and 32 (16),
// in clusters 4 and 0.
#pragma once

#include <cmath>
#include <cstdint>
#include <cuda_fp16.h>

#include "kv4_store.cuh"
#include "ptx.cuh"

namespace pasa {

// Warps of a CTA and CTAs of an SM, by the tile's rows / 8: 2 x 8 warps of 128 registers, or with 16 rows, whose
// accumulators take twice as many, 1 x 12 of 168 (16 rows x 131072 keys x 8: 145 us; 2 x 8, which spill more, 159).
__host__ __device__ constexpr int kv4_warps(int nt) { return nt == 1 ? 8 : 12; }
__host__ __device__ constexpr int kv4_ctas(int nt) { return nt == 1 ? 304 : 152; }   // on 152 SMs
constexpr int kKv4WeightsWarps = 8;
constexpr int kKv4Alone = 120 * 1024;   // dynamic shared memory with which a CTA has its SM alone
constexpr int kKv4Unit = 32;    // keys a warp takes at a time
constexpr int kKv4SegmentStart = 2;    // rounds that the start and end of a segment cost a CTA

struct Kv4Params {
  const __half* q;
  const uint8_t *k4, *v4;
  const __half *kscale, *vscale, *shift;   // shift: [B, Hkv, D] or nullptr
  const int* lengths;                      // [B] or nullptr: Sk rows in every sequence
  __half* o;
  float* lse;        // or nullptr
  float* weights;    // [B, Hkv, cap] or nullptr
  float* part_o;     // [2 gridDim.x][tile rows][D]: a CTA's first segment, and its last
  float2* part_ml;   // [2 gridDim.x][tile rows]: max (log2 units), sum
  float* lse2;       // [segments][tile rows]: log2-sum-exp2 of the shifted scores, for the weights pass
  int B, Hkv, Sq, rows, row_tiles;         // rows = Hq / Hkv * Sq query rows of a kv head
  int Sk, cap, causal;
  int len_add;       // added to lengths[] (a step call appends that many rows first)
  int ctas;          // gridDim.x of the stream-K decode
  int cluster;       // CTAs that share a segment (1 with stream-K)
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

__host__ __device__ __forceinline__ constexpr int kv4_units(int len) { return (len + kKv4Unit - 1) / kKv4Unit; }

// A segment's weight when segments are shared out: its rounds (a unit for each warp of a CTA: what
// is shared is whole rounds, so that no warp idles in the middle), and kKv4SegmentStart.
__host__ __device__ __forceinline__ constexpr int kv4_rounds(int units, int warps) { return (units + warps - 1) / warps; }
__device__ __forceinline__ int kv4_weight(int units, int warps) {
  return units == 0 ? 0 : kv4_rounds(units, warps) + kKv4SegmentStart;
}

// The weights of all sequences (per kv head and row tile), looked at by a whole warp: their sum, the
// sum of the first b, and the sequence that a place falls in. The lanes hold the first 32
// lengths and their running sums, so that a batch that small is read and scanned once. All
// weights of a call fit an int (checked on the host).
struct Kv4Lengths {
  const Kv4Params& p;
  int warps;       // of a CTA
  int len, upto;   // lane l: length l of the first 32, and their weights up to it
  __device__ __forceinline__ Kv4Lengths(const Kv4Params& params, int cta_warps) : p(params), warps(cta_warps) {
    block(0, len, upto);
  }
  __device__ __forceinline__ void block(int b0, int& l, int& sum) const {
    const int lane = threadIdx.x & 31;
    l = b0 + lane < p.B ? p.length(b0 + lane) : 0;
    sum = kv4_weight(kv4_units(l), warps);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xFFFFFFFFu, sum, d);
      if (lane >= d) sum += x;
    }
  }
  __device__ __forceinline__ int sum(int b_end) const {
    int n = 0, l, s = upto;
    for (int b0 = 0; b0 < b_end; b0 += 32) {
      if (b0 > 0) block(b0, l, s);
      n += __shfl_sync(0xFFFFFFFFu, s, min(b_end - b0, 32) - 1);
    }
    return n;
  }
  // The sequence b that `place` falls in, each sequence's weight counted per_b times; `place` becomes
  // the place inside b. place is less than the sum.
  __device__ __forceinline__ int find(int& place, int per_b, int& length) const {
    int l = len, s = upto;
    for (int b0 = 0;; b0 += 32) {
      if (b0 > 0) block(b0, l, s);
      const uint32_t past = __ballot_sync(0xFFFFFFFFu, s * per_b > place);
      if (past != 0) {
        const int lane = __ffs(past) - 1;
        length = __shfl_sync(0xFFFFFFFFu, l, lane);
        place -= (__shfl_sync(0xFFFFFFFFu, s, lane) - kv4_weight(kv4_units(length), warps)) * per_b;
        return b0 + lane;
      }
      place -= __shfl_sync(0xFFFFFFFFu, s, 31) * per_b;
    }
  }
};

// The rounds [first(c), first(c + 1)) of CTA c of `ctas`, total >= ctas >= 1: as equal as can be.
struct Kv4Share {
  unsigned base, more;   // rounds of a CTA, and how many CTAs have one more
  __device__ __forceinline__ Kv4Share(int total, int ctas)
      : base(static_cast<unsigned>(total) / ctas), more(static_cast<unsigned>(total) - base * ctas) {}
  __device__ __forceinline__ int first(unsigned c) const { return c * base + min(c, more); }
  __device__ __forceinline__ int cta_of(unsigned u) const {
    const unsigned split = more * (base + 1);
    return u < split ? u / (base + 1) : more + (u - split) / base;
  }
};

// d = A B + (c0, c1) of every output row pair: m16n8k16, fp16 in, fp32 out.
__device__ __forceinline__ void mma_f16_init(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1, float c0, float c1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%10,%11};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
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

template <bool TRANS>
__device__ __forceinline__ void ldmatrix_x4(uint32_t (&d)[4], uint32_t saddr) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3]) : "r"(saddr) : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3]) : "r"(saddr) : "memory");
}

// 16 bytes from global to shared memory, asynchronously. `policy`: what L2 does with the line.
__device__ __forceinline__ void cp_async16(uint32_t saddr, const void* g, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(saddr), "l"(g), "l"(policy)
               : "memory");
}
// Codes stream past once: they leave L2 first, so that queries, lengths and partial results stay.
__device__ __forceinline__ uint64_t evict_first_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// A warp's stage of 32 rows of codes: 16-byte chunk c (channels 32 c .. 32 c + 31) of row r at
// r * D/2 + 16 (c ^ swizzle(r)), so that the 8 rows of an 8 x 8 ldmatrix block lie in 8 different
// bank groups.
template <int D>
__device__ __forceinline__ uint32_t kv4_chunk(int row, int c) {
  return static_cast<uint32_t>(D == 128 ? row * 64 + ((c ^ ((row >> 1) & 3)) << 4) : row * 32 + ((c ^ ((row >> 2) & 1)) << 4));
}

// Start copying the codes of 32 rows to a stage; rows from `left` on are filled with zeros, not
// read. rows: this lane's first 16 bytes (16 lane past the unit's first row); stage: likewise its
// swizzled place, the same for all its chunks but for multiples of 512 bytes.
template <int D>
__device__ __forceinline__ uint32_t kv4_lane_place(int lane) { return kv4_chunk<D>(lane / (D / 32), lane % (D / 32)); }
template <int D>
__device__ __forceinline__ void kv4_fetch(uint32_t stage, const uint8_t* rows, int left, int lane, uint64_t policy) {
  constexpr int kChunks = D / 32;   // per row
  if (left >= kKv4Unit) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) cp_async16(stage + 512 * i, rows + 512 * i, policy);
  } else {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      if ((i * 32 + lane) / kChunks < left)
        cp_async16(stage + 512 * i, rows + 512 * i, policy);
      else
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(stage + 512 * i), "r"(0) : "memory");
    }
  }
}

// The scales of one row (D / 32 fp16), lane l holding row l's; 0 past the last row.
template <int D>
__device__ __forceinline__ uint2 kv4_row_scales(const __half* rows, int left, int lane) {
  uint2 s = make_uint2(0u, 0u);
  if (lane < left) {
    if constexpr (D == 128)
      s = *reinterpret_cast<const uint2*>(rows + lane * 4);
    else
      s.x = *reinterpret_cast<const uint32_t*>(rows + lane * 2);
  }
  return s;
}

// 8 query rows as S needs them, in the lanes of a warp. The scores of a group of 32 channels
// are the MMA of raw codes: a code masked out of its byte is a subnormal fp16 number, n 2^-24 or
// (the high nibble) n 2^-20, n = c + 8, so the query entries it meets are q' 2^4 or q', and the
// -8 of every code is the accumulator's start, -8 2^-20 sum q'. No instruction per value but
// the mask; the group's scale multiplies the fp32 sum. q' = q 2^e with the row's largest |q'|
// in [2^10, 2^11): exact but for entries 2^-34 below the largest.
template <int D>
struct Kv4Query {
  uint4 b[D / 32];      // per group: channels (0, 4) and (2, 6) times 16, (1, 5), (3, 7) of the lane's 8
  float start[D / 32];  // of row g: -8 2^-20 sum q'
  float factor;         // of row g: scores to log2 units: scale log2(e) 2^(20 - e)
  // The raw rows, n of 8: to be asked for ahead of the codes, whose first burst fills the memory system.
  static __device__ __forceinline__ void raw(uint4 (&x)[D / 32], const __half* rows, int n, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
      x[w] = make_uint4(0u, 0u, 0u, 0u);
      if (g < n) x[w] = *reinterpret_cast<const uint4*>(rows + g * D + 32 * w + 8 * t);
    }
  }
  __device__ __forceinline__ void prepare(const uint4 (&x)[D / 32], float scale_log2) {
    __half2 m2 = __float2half2_rn(0.0f);
#pragma unroll
    for (int w = 0; w < D / 32; ++w)
      m2 = __hmax2_nan(m2, __hmax2_nan(__hmax2_nan(__habs2(bits_h2(x[w].x)), __habs2(bits_h2(x[w].y))),
                                       __hmax2_nan(__habs2(bits_h2(x[w].z)), __habs2(bits_h2(x[w].w)))));
    __half m1 = __hmax_nan(__low2half(m2), __high2half(m2));
    m1 = __hmax_nan(m1, __shfl_xor_sync(0xFFFFFFFFu, m1, 1));
    m1 = __hmax_nan(m1, __shfl_xor_sync(0xFFFFFFFFu, m1, 2));
    const float m = __half2float(m1);
    // a row that is all 0, or not finite, is left as it is
    const int e = m > 0.0f && m <= 65504.0f ? 137 - static_cast<int>(__float_as_uint(m) >> 23) : 0;
    const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    factor = scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + 20 - e) << 23);
    const __half2 sixteen = __float2half2_rn(16.0f);
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
      const uint32_t in[4] = {x[w].x, x[w].y, x[w].z, x[w].w};
      uint32_t h[4];
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 v = __half22float2(bits_h2(in[i]));
        v.x *= up, v.y *= up;
        const __half2 r = __float22half2_rn(v);
        v = __half22float2(r);
        sum += v.x + v.y;
        h[i] = h2_bits(r);
      }
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
      start[w] = sum * (-8.0f / 1048576.0f);
      b[w].x = h2_bits(__hmul2(bits_h2(__byte_perm(h[0], h[2], 0x5410)), sixteen));
      b[w].y = h2_bits(__hmul2(bits_h2(__byte_perm(h[1], h[3], 0x5410)), sixteen));
      b[w].z = __byte_perm(h[0], h[2], 0x7632);
      b[w].w = __byte_perm(h[1], h[3], 0x7632);
    }
  }
  // A value of row g as the values of rows 2t and 2t + 1, the columns of an output fragment.
  static __device__ __forceinline__ float2 columns(float x, int lane) {
    return make_float2(__shfl_sync(0xFFFFFFFFu, x, 8 * (lane & 3)), __shfl_sync(0xFFFFFFFFu, x, 8 * (lane & 3) + 4));
  }
};

// 8 rows in shared memory as S^T needs them, for the warps of a CTA to share.
template <int D>
struct __align__(16) Kv4QueryShared {
  uint4 b[D / 32][32];
  float2 init[D / 32][32];
  float2 factor[32];
  __device__ __forceinline__ void put(const Kv4Query<D>& q, int lane) {
#pragma unroll
    for (int w = 0; w < D / 32; ++w) b[w][lane] = q.b[w], init[w][lane] = Kv4Query<D>::columns(q.start[w], lane);
    factor[lane] = Kv4Query<D>::columns(q.factor, lane);
  }
};

// 16 rows in shared memory as S = Q K'^T needs them: the A operands of a group's two MMAs.
template <int D>
struct __align__(16) Kv4Query16 {
  uint32_t a[D / 32][2][32][4];
  float start[D / 32][32][2];    // rows g, g + 8
  float factor[32][2];
  __device__ __forceinline__ void put(const Kv4Query<D>& q, int tile, int lane) {
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
      a[w][0][lane][tile] = q.b[w].x, a[w][0][lane][2 + tile] = q.b[w].y;
      a[w][1][lane][tile] = q.b[w].z, a[w][1][lane][2 + tile] = q.b[w].w;
      start[w][lane][tile] = q.start[w];
    }
    factor[lane][tile] = q.factor;
  }
};

// S^T (unscaled) of 16 keys and 8 rows, group w's part added to acc (set where w is 0). ka, kb:
// the lane's 8 codes of keys g and g + 8 in the group; sa, sb: their scales.
__device__ __forceinline__ void kv4_score_group(float (&acc)[4], int w, uint32_t ka, uint32_t kb, float sa, float sb,
                                                const uint4& qb, const float2& init) {
  const uint32_t lo = 0x000F000Fu, hi = 0x00F000F0u;
  const uint32_t a8 = ka >> 8, b8 = kb >> 8;
  float d[4];
  mma_f16_init(d, ka & lo, kb & lo, a8 & lo, b8 & lo, qb.x, qb.y, init.x, init.y);
  mma_f16(d, ka & hi, kb & hi, a8 & hi, b8 & hi, qb.z, qb.w);
  acc[0] = w == 0 ? sa * d[0] : fmaf(sa, d[0], acc[0]);
  acc[1] = w == 0 ? sa * d[1] : fmaf(sa, d[1], acc[1]);
  acc[2] = w == 0 ? sb * d[2] : fmaf(sb, d[2], acc[2]);
  acc[3] = w == 0 ? sb * d[3] : fmaf(sb, d[3], acc[3]);
}

// S (unscaled) of 16 rows (g and g + 8) and the keys 2t and 2t + 1 of 8, group w's part; k: the
// lane's 8 codes of key g, s0, s1: the scales of the two keys.
__device__ __forceinline__ void kv4_score_group16(float (&acc)[4], int w, uint32_t k, float s0, float s1, const uint4& qa,
                                                  const uint4& qb, const float2& start) {
  const uint32_t lo = 0x000F000Fu, hi = 0x00F000F0u;
  const uint32_t k8 = k >> 8;
  float d[4];
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%11,%11};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(qa.x), "r"(qa.y), "r"(qa.z), "r"(qa.w), "r"(k & lo), "r"(k8 & lo), "f"(start.x), "f"(start.y));
  mma_f16(d, qb.x, qb.y, qb.z, qb.w, k & hi, k8 & hi);
  if (w == 0) {
    fmul2(acc[0], acc[1], d[0], d[1], s0, s1);
    fmul2(acc[2], acc[3], d[2], d[3], s0, s1);
  } else {
    ffma2(acc[0], acc[1], d[0], d[1], s0, s1, acc[0], acc[1]);
    ffma2(acc[2], acc[3], d[2], d[3], s0, s1, acc[2], acc[3]);
  }
}

// One stage of a warp: 32 rows of key and value codes and their scales. Where a lane needs keys by
// pairs (8 blk + 2 t, + 1 for blk = 0 .. 3), the scales are [group][8 t + 2 blk + key % 2]: the
// values' as fp16, and with 16 query rows (PAIRS) the keys' as fp32; else those are rows.
template <int D, bool VALUES>
struct __align__(128) Kv4Stage {
  uint8_t k[kKv4Unit * D / 2];
  uint8_t v[VALUES ? kKv4Unit * D / 2 : 16];
  float ks[kKv4Unit * D / 32];
  __half vs[D / 32][kKv4Unit];
};

template <int D, bool VALUES, bool PAIRS>
__device__ __forceinline__ void kv4_put_scales(Kv4Stage<D, VALUES>& st, uint2 ks, uint2 vs, int lane) {
  const int at = (lane >> 1 & 3) * 8 + (lane >> 3) * 2 + (lane & 1);
  const float2 a = __half22float2(bits_h2(ks.x)), b = __half22float2(bits_h2(ks.y));
  if constexpr (PAIRS) {
    st.ks[at] = a.x, st.ks[32 + at] = a.y;
    if constexpr (D == 128) st.ks[64 + at] = b.x, st.ks[96 + at] = b.y;
  } else if constexpr (D == 128) {
    *reinterpret_cast<float4*>(&st.ks[4 * lane]) = make_float4(a.x, a.y, b.x, b.y);
  } else {
    *reinterpret_cast<float2*>(&st.ks[2 * lane]) = a;
  }
  if constexpr (VALUES) {
    st.vs[0][at] = __low2half(bits_h2(vs.x));
    st.vs[1][at] = __high2half(bits_h2(vs.x));
    if constexpr (D == 128) {
      st.vs[2][at] = __low2half(bits_h2(vs.y));
      st.vs[3][at] = __high2half(bits_h2(vs.y));
    }
  }
}

// The codes of keys 16 h + g (ka) and 16 h + 8 + g (kb) from a stage: word w the lane's 8
// channels 32 w + 8 t ... `base`: the stage's key codes + kv4_key_place.
template <int D>
__device__ __forceinline__ uint32_t kv4_key_place(int lane) {
  return D == 128 ? kv4_chunk<D>(lane & 7, lane >> 3) : kv4_chunk<D>(8 * (lane >> 4) + (lane & 7), (lane >> 3) & 1);
}
template <int D>
__device__ __forceinline__ void kv4_take_keys(uint32_t (&ka)[D / 32], uint32_t (&kb)[D / 32], uint32_t base, int h) {
  if constexpr (D == 128) {   // matrix j: chunk j of 8 rows
    ldmatrix_x4<false>(ka, base + 1024 * h);
    ldmatrix_x4<false>(kb, base + 1024 * h + 512);
  } else {                    // matrix j: chunk j % 2 of rows 8 (j / 2) ..
    uint32_t x[4];
    ldmatrix_x4<false>(x, base + 512 * h);
    ka[0] = x[0], ka[1] = x[1], kb[0] = x[2], kb[1] = x[3];
  }
}
template <int D>
__device__ __forceinline__ void kv4_take_scales(float (&s)[D / 32], const float* row) {
  if constexpr (D == 128) {
    const float4 x = *reinterpret_cast<const float4*>(row);
    s[0] = x.x, s[1] = x.y, s[2] = x.z, s[3] = x.w;
  } else {
    const float2 x = *reinterpret_cast<const float2*>(row);
    s[0] = x.x, s[1] = x.y;
  }
}

// Finish a row: O and LSE from sum, max and the unnormalised O held in shared or global memory.
__device__ __forceinline__ float kv4_lse(float m, float l, float offset) {
  return l == 0.0f ? -INFINITY : 0.69314718055994531f * (m + log2f(l)) + offset;
}

constexpr float kKv4NoKey = -3.0e38f;   // a running maximum before the first key: below every score

template <int D, int NT>
struct Kv4Smem {
  union {
    Kv4Stage<D, true> stage[2][kv4_warps(NT)];
    float o[kv4_warps(NT)][NT * 8][D + 4];   // when the stages are empty
  };
  Kv4Query16<D> q;                       // NT = 2
  float sum[NT * 8][D];                  // the CTA's O, maxima and sums, read by its cluster
  float2 sum_ml[NT * 8];
  float2 ml[kv4_warps(NT)][NT * 8];
  float offset[NT * 8];
  int limit[NT * 8];                     // keys a row sees
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

// Write channels ch .. ch + 3 of a row, and with channel 0 its log-sum-exps.
template <int D>
__device__ __forceinline__ void kv4_finish(const Kv4Params& p, long long out, long long lse2_at, int ch, float4 x, float mm,
                                           float ll, float offset) {
  const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
  const __half2 a = __floats2half2_rn(x.x * inv, x.y * inv), b = __floats2half2_rn(x.z * inv, x.w * inv);
  *reinterpret_cast<uint2*>(p.o + out * D + ch) = make_uint2(h2_bits(a), h2_bits(b));
  if (ch == 0) {
    if (p.lse) p.lse[out] = kv4_lse(mm, ll, offset);
    if (p.weights) p.lse2[lse2_at] = ll == 0.0f ? INFINITY : mm + log2f(ll);
  }
}

template <int D, int NT, bool STREAM_K>
__global__ void __launch_bounds__(kv4_warps(NT) * 32, kv4_ctas(NT) / 152) kv4_decode_kernel(Kv4Params p) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  Kv4Smem<D, NT>& sm = *reinterpret_cast<Kv4Smem<D, NT>*>(smem_raw);
  constexpr int kRows = NT * 8;
  constexpr int kWarps = kv4_warps(NT);
  constexpr int kThreads = kWarps * 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int rank = STREAM_K ? 0 : static_cast<int>(blockIdx.x % p.cluster);
  griddep_launch_dependents();
  const uint64_t policy = evict_first_policy();

  // this CTA's segments: (b, h, row tile) in order, its rounds in all, and the first one's number
  int todo = 0, b = 0, r0 = 0, n_units = 0, len = 0;
  int in_b = 0;   // segment inside sequence b: h * row_tiles + row tile
  const int per_b = p.Hkv * p.row_tiles;
  if (STREAM_K) {
    const Kv4Lengths lengths(p, kWarps);
    const int total = lengths.sum(p.B) * per_b;
    const int ctas = min(total, static_cast<int>(gridDim.x));
    if (static_cast<int>(blockIdx.x) >= ctas) {
      griddep_wait();   // every CTA: what is behind this kernel waits for this kernel only
      return;
    }
    const Kv4Share share(total, ctas);
    int place = share.first(blockIdx.x);
    todo = share.first(blockIdx.x + 1) - place;
    b = lengths.find(place, per_b, len);
    n_units = kv4_units(len);
    const int weight = kv4_weight(n_units, kWarps);
    in_b = place / weight;
    r0 = place - in_b * weight - kKv4SegmentStart;   // its first rounds stand for its start
  } else {
    const int seg = blockIdx.x / p.cluster;
    b = seg / per_b;
    in_b = seg - b * per_b;
    len = p.length(b);
    n_units = kv4_units(len);
    todo = n_units;
  }

  griddep_wait();   // the rows that a step's append stores; nothing so far is its
  for (int nth = 0;; nth = 1) {   // 0: the CTA's first segment
    const long long bh = static_cast<long long>(b) * p.Hkv + in_b / p.row_tiles;
    const int row0 = in_b % p.row_tiles * kRows;
    const int n_rows = min(kRows, p.rows - row0);
    int u0 = 0, u1 = n_units;
    if (STREAM_K) {
      const int r1 = min(kv4_rounds(n_units, kWarps), r0 + todo);
      todo -= r1 - r0;
      u0 = max(0, r0) * kWarps;
      u1 = min(n_units, r1 * kWarps);
      if (u0 >= u1) return;   // the range ends in what a segment's start weighs
    }
    const int u_step = STREAM_K ? kWarps : kWarps * p.cluster;

    // ---- the warp's share of units u0 .. u1 ----
    int u = u0 + rank * kWarps + warp;
    const uint32_t stage0 = smem_u32(&sm.stage[0][warp]);
    constexpr uint32_t kStageBytes = sizeof(Kv4Stage<D, true>) * kWarps, kValues = kKv4Unit * D / 2;
    uint2 ks = make_uint2(0u, 0u), vs = make_uint2(0u, 0u);   // row scales of the unit last fetched
    auto fetch = [&](int unit, uint32_t stage) {
      if (unit < u1) {
        const long long row = bh * p.cap + static_cast<long long>(unit) * kKv4Unit;
        const int left = len - unit * kKv4Unit;
        const uint32_t place = stage + kv4_lane_place<D>(lane);
        kv4_fetch<D>(place, p.k4 + row * (D / 2) + lane * 16, left, lane, policy);
        kv4_fetch<D>(place + kValues, p.v4 + row * (D / 2) + lane * 16, left, lane, policy);
        ks = kv4_row_scales<D>(p.kscale + row * (D / 32), left, lane);
        vs = kv4_row_scales<D>(p.vscale + row * (D / 32), left, lane);
      }
      cp_async_commit();
    };
    // the queries: NT = 1 in registers, else in shared memory, 8 rows per warp
    Kv4Query<D> q;
    {
      uint4 raw[D / 32];
      const int tile = NT == 1 ? 0 : warp;
      if (tile < NT) Kv4Query<D>::raw(raw, p.q + (bh * p.rows + row0 + tile * 8) * D, n_rows - tile * 8, lane);
      fetch(u, stage0);
      if (tile < NT) q.prepare(raw, p.scale_log2);
      if (NT == 2 && tile < NT) sm.q.put(q, tile, lane);
    }
    float2 init[D / 32], factor;
    if constexpr (NT == 1) {
#pragma unroll
      for (int w = 0; w < D / 32; ++w) init[w] = Kv4Query<D>::columns(q.start[w], lane);
      factor = Kv4Query<D>::columns(q.factor, lane);
    }
    if (threadIdx.x < kRows) sm.limit[threadIdx.x] = p.limit(row0 + threadIdx.x, len);
    const bool whole = u0 == 0 && u1 == n_units;   // the CTA, or its cluster, has all of the segment
    if (whole && rank == 0 && p.lse)
      for (int r = warp; r < n_rows; r += kWarps) {
        const float off = kv4_offset<D>(p, bh, row0 + r, lane);
        if (lane == 0) sm.offset[r] = off;
      }
    __syncthreads();
    if constexpr (NT == 2) factor = make_float2(sm.q.factor[lane][0], sm.q.factor[lane][1]);
    // O: with 8 rows O^T (channels along g, the lane's rows 2t, 2t + 1), with 16 O (its rows g, g + 8)
    constexpr int kTiles = NT == 1 ? D / 16 : D / 8;
    float o[kTiles][4];
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.0f;
    // of the lane's two rows; with 16 rows the sums of even and odd keys apart
    float m[2] = {kKv4NoKey, kKv4NoKey}, l[2 * NT] = {};
    const int all_see = p.causal ? max(0, len - p.Sq + 1) : len;   // keys that every row sees
    uint32_t odd = 0;   // the stage at hand
    for (; u < u1; u += u_step) {
      const int key0 = u * kKv4Unit;
      auto& st = sm.stage[odd][warp];
      const uint32_t here = stage0 + odd * kStageBytes;
      cp_async_wait<0>();
      kv4_put_scales<D, true, NT == 2>(st, ks, vs, lane);
      __syncwarp();   // the stage is there, and every lane is done with the other one
      odd ^= 1;
      fetch(u + u_step, stage0 + odd * kStageBytes);
      // s[i]: of the lane's rows and 2 keys; NT = 1: i = half h, keys 16 h + g (elements 0, 1: rows 2t,
      // 2t + 1) and 16 h + 8 + g (2, 3); NT = 2: i = blk, keys 8 blk + 2 t, + 1 of row g (0, 1) and g + 8
      float s[2 * NT][4];
      if constexpr (NT == 1) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t ka[D / 32], kb[D / 32];
          kv4_take_keys<D>(ka, kb, here + kv4_key_place<D>(lane), h);
          float sa[D / 32], sb[D / 32];
          kv4_take_scales<D>(sa, &st.ks[(16 * h + g) * (D / 32)]);
          kv4_take_scales<D>(sb, &st.ks[(16 * h + 8 + g) * (D / 32)]);
#pragma unroll
          for (int w = 0; w < D / 32; ++w) kv4_score_group(s[h], w, ka[w], kb[w], sa[w], sb[w], q.b[w], init[w]);
        }
      } else {
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          const uint4 qa = *reinterpret_cast<const uint4*>(sm.q.a[w][0][lane]);
          const uint4 qb = *reinterpret_cast<const uint4*>(sm.q.a[w][1][lane]);
          const float2 start = *reinterpret_cast<const float2*>(sm.q.start[w][lane]);
          uint32_t k[4];   // key 8 blk + g, channels 32 w + 8 t ..
          ldmatrix_x4<false>(k, (here + kv4_chunk<D>(lane, 0)) ^ (w << 4));
          float sc[8];
          *reinterpret_cast<float4*>(sc) = *reinterpret_cast<const float4*>(&st.ks[32 * w + 8 * t]);
          *reinterpret_cast<float4*>(sc + 4) = *reinterpret_cast<const float4*>(&st.ks[32 * w + 8 * t + 4]);
#pragma unroll
          for (int blk = 0; blk < 4; ++blk)
            kv4_score_group16(s[blk], w, k[blk], sc[2 * blk], sc[2 * blk + 1], qa, qb, start);
        }
      }
      if (key0 + kKv4Unit > all_see) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int lim = sm.limit[NT == 1 ? 2 * t + c : g + 8 * c] - key0 - (NT == 1 ? g : 2 * t);
#pragma unroll
          for (int i = 0; i < 2 * NT; ++i) {
            if (NT == 1) {
              if (16 * i >= lim) s[i][c] = -INFINITY;
              if (16 * i + 8 >= lim) s[i][2 + c] = -INFINITY;
            } else {
              if (8 * i >= lim) s[i][2 * c] = -INFINITY;
              if (8 * i + 1 >= lim) s[i][2 * c + 1] = -INFINITY;
            }
          }
        }
      }
      // the reference a row's exponentials are taken against moves only when a score passes it
      // by more than 8 (log2 units): P stays below 2^8, and most units need no reduction
      float mx[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        mx[c] = -INFINITY;
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i)
          mx[c] = fmaxf(mx[c], NT == 1 ? fmaxf(s[i][c], s[i][2 + c]) : fmaxf(s[i][2 * c], s[i][2 * c + 1]));
        mx[c] *= c ? factor.y : factor.x;
      }
      if (__any_sync(0xFFFFFFFFu, mx[0] > m[0] + 8.0f || mx[1] > m[1] + 8.0f)) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float x = mx[c];   // over the lanes that share the row
#pragma unroll
          for (int d = NT == 1 ? 4 : 1; d < (NT == 1 ? 32 : 4); d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, d));
          x = fmaxf(x, m[c]);
          const float f = ex2_approx(m[c] - x);
          m[c] = x;
          if (NT == 1) l[c] *= f; else l[NT * c] *= f, l[NT * c + NT - 1] *= f;
#pragma unroll
          for (int i = 0; i < kTiles; ++i) {
            o[i][NT == 1 ? c : 2 * c] *= f;
            o[i][NT == 1 ? 2 + c : 2 * c + 1] *= f;
          }
        }
      }
      // P in fp16, NT = 1: P^T as the B operand (keys and rows change places: movmatrix), NT = 2: as A
      uint32_t pf[2][2 * NT];
#pragma unroll
      for (int i = 0; i < 2 * NT; ++i) {
        // pairs: NT = 1 (row 2t, row 2t + 1), NT = 2 two keys of row g, then of row g + 8
        float e[4];
        if constexpr (NT == 1) {
          ffma2(e[0], e[1], s[i][0], s[i][1], factor.x, factor.y, -m[0], -m[1]);
          ffma2(e[2], e[3], s[i][2], s[i][3], factor.x, factor.y, -m[0], -m[1]);
        } else {
          ffma2(e[0], e[1], s[i][0], s[i][1], factor.x, factor.x, -m[0], -m[0]);
          ffma2(e[2], e[3], s[i][2], s[i][3], factor.y, factor.y, -m[1], -m[1]);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) e[c] = ex2_approx(e[c]);
        if constexpr (NT == 1) {
          fadd2(l[0], l[1], l[0], l[1], e[0], e[1]);
          fadd2(l[0], l[1], l[0], l[1], e[2], e[3]);
        } else {
          fadd2(l[0], l[1], l[0], l[1], e[0], e[1]);
          fadd2(l[2], l[3], l[2], l[3], e[2], e[3]);
        }
        const uint32_t p01 = h2_bits(__floats2half2_rn(e[0], e[1])), p23 = h2_bits(__floats2half2_rn(e[2], e[3]));
        if constexpr (NT == 1) {
          pf[i][0] = movmatrix(p01);
          pf[i][1] = movmatrix(p23);
        } else {
          pf[i / 2][2 * (i % 2)] = p01;
          pf[i / 2][2 * (i % 2) + 1] = p23;
        }
      }
      // O += P V, a group of 32 channels at a time: a transposed 8 x 8 block of 16-bit words is 4
      // channels (4 g ..) of the two keys 8 blk + 2 t, + 1
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        uint32_t v[4];
        ldmatrix_x4<true>(v, (here + kValues + kv4_chunk<D>(lane, 0)) ^ (j << 4));   // chunk j: stages are 128-byte aligned
        const uint4 sv = *reinterpret_cast<const uint4*>(&st.vs[j][8 * t]);
        const uint32_t s2[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          __half2 a[4], c[4];
          kv4_expand(v[2 * h], bits_h2(s2[2 * h]), a);
          kv4_expand(v[2 * h + 1], bits_h2(s2[2 * h + 1]), c);
          if constexpr (NT == 1) {
            mma_f16(o[2 * j], h2_bits(a[0]), h2_bits(a[1]), h2_bits(c[0]), h2_bits(c[1]), pf[h][0], pf[h][1]);
            mma_f16(o[2 * j + 1], h2_bits(a[2]), h2_bits(a[3]), h2_bits(c[2]), h2_bits(c[3]), pf[h][0], pf[h][1]);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)   // channels 32 j + 4 n + i, n the output's column
              mma_f16(o[4 * j + i], pf[h][0], pf[h][1], pf[h][2], pf[h][3], h2_bits(a[i]), h2_bits(c[i]));
          }
        }
      }
    }
    __syncthreads();   // no stage is read or written any more: their space is free

    // ---- join the warps ----
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float x = NT == 1 ? l[c] : l[NT * c] + l[NT * c + NT - 1];
#pragma unroll
      for (int d = NT == 1 ? 4 : 1; d < (NT == 1 ? 32 : 4); d <<= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
      const int r = NT == 1 ? 2 * t + c : g + 8 * c;
      if ((NT == 1 ? g : t) == 0) sm.ml[warp][r] = make_float2(m[c], x);
      // 4 channels at a time; a row stride of 4 floats past a multiple of 32 spreads the quarter
      // warps' rows over the banks
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        float* to = &sm.o[warp][r][32 * j];
        if constexpr (NT == 1) {
          *reinterpret_cast<float4*>(to + 4 * g) = make_float4(o[2 * j][c], o[2 * j][2 + c], o[2 * j + 1][c], o[2 * j + 1][2 + c]);
        } else {
#pragma unroll
          for (int n = 0; n < 2; ++n)
            *reinterpret_cast<float4*>(to + 8 * t + 4 * n) =
                make_float4(o[4 * j][2 * c + n], o[4 * j + 1][2 * c + n], o[4 * j + 2][2 * c + n], o[4 * j + 3][2 * c + n]);
        }
      }
    }
    __syncthreads();
    const long long seg = static_cast<long long>(b) * per_b + in_b;
    const long long out0 = bh * p.rows + row0;
    const bool alone = STREAM_K || p.cluster == 1;
    // a thread: 4 channels of a row, the row's maximum and sum with them
    for (int idx = threadIdx.x; idx < n_rows * (D / 4); idx += kThreads) {
      const int r = idx / (D / 4), ch = idx % (D / 4) * 4;
      float2 ml[kWarps];
      float mm = kKv4NoKey, ll = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        ml[w] = sm.ml[w][r];
        mm = fmaxf(mm, ml[w].x);
      }
      float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2_approx(ml[w].x - mm);   // a warp without a key of this row has sum 0
        const float4 v = *reinterpret_cast<const float4*>(&sm.o[w][r][ch]);
        ll = fmaf(f, ml[w].y, ll);
        x.x = fmaf(f, v.x, x.x), x.y = fmaf(f, v.y, x.y), x.z = fmaf(f, v.z, x.z), x.w = fmaf(f, v.w, x.w);
      }
      if (!alone) {
        *reinterpret_cast<float4*>(&sm.sum[r][ch]) = x;
        if (ch == 0) sm.sum_ml[r] = make_float2(mm, ll);
      } else if (whole) {
        kv4_finish<D>(p, out0 + r, seg * kRows + r, ch, x, mm, ll, sm.offset[r]);
      } else {
        const long long slot = (2 * blockIdx.x + nth) * kRows + r;   // only its first and last are shared
        *reinterpret_cast<float4*>(p.part_o + slot * D + ch) = x;
        if (ch == 0) p.part_ml[slot] = make_float2(mm, ll);
      }
    }
    if (!alone) {
      cluster_sync_all();
      for (int idx = threadIdx.x * p.cluster + rank; idx < n_rows * (D / 4); idx += kThreads * p.cluster) {
        const int r = idx / (D / 4), ch = idx % (D / 4) * 4;
        float2 ml[8];
        float4 v[8];
        float mm = kKv4NoKey, ll = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) {   // clusters are of 8 at most
          ml[w] = make_float2(kKv4NoKey, 0.0f), v[w] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (w < p.cluster) {
            ml[w] = ld_cluster_float2(mapa_shared(smem_u32(&sm.sum_ml[r]), w));
            v[w] = ld_cluster_float4(mapa_shared(smem_u32(&sm.sum[r][ch]), w));
          }
        }
        const float off = ch == 0 ? ld_shared_cluster_f32(mapa_shared(smem_u32(&sm.offset[r]), 0)) : 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) mm = fmaxf(mm, ml[w].x);
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          const float f = ex2_approx(ml[w].x - mm);
          ll = fmaf(f, ml[w].y, ll);
          x.x = fmaf(f, v[w].x, x.x), x.y = fmaf(f, v[w].y, x.y), x.z = fmaf(f, v[w].z, x.z), x.w = fmaf(f, v[w].w, x.w);
        }
        kv4_finish<D>(p, out0 + r, seg * kRows + r, ch, x, mm, ll, off);
      }
    }
    if (!STREAM_K) {
      if (!alone) cluster_sync_all();   // the others have read this CTA's sums
      return;
    }
    // ---- next segment ----
    if (todo <= 0) return;
    r0 = -kKv4SegmentStart;
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
  __shared__ float so[8][D], factor[kv4_ctas(1)];
  __shared__ float s_m[8], s_l[8], s_off;
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long seg = blockIdx.x;
  const long long per_b = static_cast<long long>(p.Hkv) * p.row_tiles;
  const int b = static_cast<int>(seg / per_b);
  const long long in_b = seg % per_b;
  const long long bh = static_cast<long long>(b) * p.Hkv + in_b / p.row_tiles;
  const int r = blockIdx.y, row = static_cast<int>(in_b % p.row_tiles) * tile_rows + r;
  const int warps = kv4_warps(tile_rows / 8);
  const Kv4Lengths lengths(p, warps);
  // every CTA waits for the decode, also those without work: a kernel behind this one waits for
  // this one only
  if (row >= p.rows) {
    griddep_wait();
    return;
  }
  const long long out = bh * p.rows + row;
  const int n_units = kv4_units(p.length(b));
  if (n_units == 0) {
    griddep_wait();
    if (threadIdx.x < D) p.o[out * D + threadIdx.x] = __float2half_rn(0.0f);
    if (threadIdx.x == 0) {
      if (p.lse) p.lse[out] = -INFINITY;
      if (p.weights) p.lse2[seg * tile_rows + r] = INFINITY;
    }
    return;
  }
  const int weight = kv4_weight(n_units, warps);
  const int total = lengths.sum(p.B) * static_cast<int>(per_b);
  const Kv4Share share(total, min(total, p.ctas));
  const int t0 = lengths.sum(b) * static_cast<int>(per_b) + static_cast<int>(in_b) * weight;
  const int c0 = share.cta_of(t0 + kKv4SegmentStart), n = share.cta_of(t0 + weight - 1) - c0 + 1;
  if (n == 1) {   // finished where it was computed
    griddep_wait();
    return;
  }
  if (warp == 0) {
    const float off = kv4_offset<D>(p, bh, row, lane);
    if (lane == 0) s_off = off;
  }
  griddep_wait();   // the partials
  // every partial's max and sum at once, then its factor
  constexpr int kMine = (kv4_ctas(1) + 255) / 256;
  // the row's partial of CTA c0 + i: that of its first segment, but c0 may have begun with another one
  const int begun = share.first(c0) < t0 ? 1 : 0;
  auto slot = [&](int i) { return (2ll * (c0 + i) + (i == 0 ? begun : 0)) * tile_rows + r; };
  float2 ml[kMine];
  float mm = kKv4NoKey;
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int c = i * 256 + threadIdx.x;
    ml[i] = c < n ? p.part_ml[slot(c)] : make_float2(kKv4NoKey, 0.0f);
    mm = fmaxf(mm, ml[i].x);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xFFFFFFFFu, mm, d));
  if (lane == 0) s_m[warp] = mm;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) mm = fmaxf(mm, s_m[w]);
  float ll = 0.0f;
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int c = i * 256 + threadIdx.x;
    const float f = ex2_approx(ml[i].x - mm);
    if (c < n) factor[c] = f;
    ll = fmaf(f, ml[i].y, ll);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) ll += __shfl_xor_sync(0xFFFFFFFFu, ll, d);
  if (lane == 0) s_l[warp] = ll;
  __syncthreads();
  float acc[D / 32];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) acc[e] = 0.0f;
  const float* part = p.part_o + lane * (D / 32);
#pragma unroll 4
  for (int c = warp; c < n; c += 8) {
    const float f = factor[c];
    if constexpr (D == 128) {
      const float4 x = *reinterpret_cast<const float4*>(part + slot(c) * D);
      acc[0] = fmaf(f, x.x, acc[0]), acc[1] = fmaf(f, x.y, acc[1]);
      acc[2] = fmaf(f, x.z, acc[2]), acc[3] = fmaf(f, x.w, acc[3]);
    } else {
      const float2 x = *reinterpret_cast<const float2*>(part + slot(c) * D);
      acc[0] = fmaf(f, x.x, acc[0]), acc[1] = fmaf(f, x.y, acc[1]);
    }
  }
#pragma unroll
  for (int e = 0; e < D / 32; ++e) so[warp][lane * (D / 32) + e] = acc[e];
  __syncthreads();
  ll = 0.0f;
#pragma unroll
  for (int w = 0; w < 8; ++w) ll += s_l[w];
  if (threadIdx.x < D) {
    float x = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) x += so[w][threadIdx.x];
    p.o[out * D + threadIdx.x] = __float2half_rn(ll == 0.0f ? 0.0f : x / ll);
  }
  if (threadIdx.x == 0) {
    if (p.lse) p.lse[out] = kv4_lse(mm, ll, s_off);
    if (p.weights) p.lse2[seg * tile_rows + r] = ll == 0.0f ? INFINITY : mm + log2f(ll);
  }
}

// weights[b, h, key] += sum over the kv head's rows of softmax(scale * q K'^T)[row, key], from
// the rows' log-sum-exps that the decode left in lse2: the scores are computed again from the
// key codes (half of the cache's bytes), which needs no buffer of rows x keys scores. One warp
// per 32-key unit, each weight summed and stored by one lane: the same order every time.
template <int D>
struct Kv4WeightsSmem {
  Kv4Stage<D, false> stage[2][kKv4WeightsWarps];
  float ref[128];            // a row's log2-sum-exp2
  int limit[128];
  Kv4QueryShared<D> q[16];   // as many as the rows have tiles of 8
};
static_assert(sizeof(Kv4WeightsSmem<128>) <= kKv4Alone && 2 * sizeof(Kv4WeightsSmem<128>) <= 227 * 1024);

template <int D, bool ALONE>
__global__ void __launch_bounds__(kKv4WeightsWarps * 32, ALONE ? 1 : 2) kv4_weights_kernel(Kv4Params p, int tile_rows) {
  // 16-key halves of a unit that go side by side: two take 185 registers, and with two CTAs per SM they spill
  // (8 sequences x 131072 keys, 7 rows: 204 us against 173)
  constexpr int kSide = ALONE ? 2 : 1;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  Kv4WeightsSmem<D>& sm = *reinterpret_cast<Kv4WeightsSmem<D>*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const Kv4Lengths lengths(p, kKv4WeightsWarps);
  const int total = lengths.sum(p.B) * p.Hkv;
  const int ctas = min(total, static_cast<int>(gridDim.x));
  if (static_cast<int>(blockIdx.x) >= ctas) {
    griddep_wait();
    return;
  }
  const Kv4Share share(total, ctas);
  int place = share.first(blockIdx.x), todo = share.first(blockIdx.x + 1) - place, len;
  int b = lengths.find(place, p.Hkv, len);
  int n_units = kv4_units(len);
  int h = place / kv4_weight(n_units, kKv4WeightsWarps);
  int r0 = place - h * kv4_weight(n_units, kKv4WeightsWarps) - kKv4SegmentStart;
  griddep_wait();   // lse2
  const uint64_t policy = evict_first_policy();
  while (true) {
    const long long bh = static_cast<long long>(b) * p.Hkv + h;
    const int r1 = min(kv4_rounds(n_units, kKv4WeightsWarps), r0 + todo);
    todo -= r1 - r0;
    const int u0 = max(0, r0) * kKv4WeightsWarps, u1 = min(n_units, r1 * kKv4WeightsWarps);
    if (u0 >= u1) return;
    const uint8_t* k4 = p.k4 + bh * p.cap * (D / 2);
    const __half* kscale = p.kscale + bh * p.cap * (D / 32);
    const uint32_t stage0 = smem_u32(&sm.stage[0][warp]);
    constexpr uint32_t kStageBytes = sizeof(Kv4Stage<D, false>) * kKv4WeightsWarps;
    uint2 ks = make_uint2(0u, 0u);
    auto fetch = [&](int unit, uint32_t stage) {
      if (unit < u1) {
        const long long key = static_cast<long long>(unit) * kKv4Unit;
        const int left = len - unit * kKv4Unit;
        kv4_fetch<D>(stage + kv4_lane_place<D>(lane), k4 + key * (D / 2) + lane * 16, left, lane, policy);
        ks = kv4_row_scales<D>(kscale + key * (D / 32), left, lane);
      }
      cp_async_commit();
    };
    int u = u0 + warp;
    for (int i = warp; i * 8 < p.rows; i += kKv4WeightsWarps) {
      Kv4Query<D> q;
      uint4 raw[D / 32];
      Kv4Query<D>::raw(raw, p.q + (bh * p.rows + i * 8) * D, p.rows - i * 8, lane);
      if (i == warp) fetch(u, stage0);
      q.prepare(raw, p.scale_log2);
      sm.q[i].put(q, lane);
    }
    if (warp * 8 >= p.rows) fetch(u, stage0);
    for (int r = threadIdx.x; r < (p.rows + 7) / 8 * 8; r += kKv4WeightsWarps * 32) {
      // a row past the last, or without a key, weighs nothing
      sm.ref[r] = r < p.rows ? p.lse2[(bh * p.row_tiles + r / tile_rows) * tile_rows + r % tile_rows] : INFINITY;
      sm.limit[r] = p.limit(r, len);
    }
    __syncthreads();
    const int all_see = p.causal ? max(0, len - p.Sq + 1) : len;
    uint32_t odd = 0;
    for (; u < u1; u += kKv4WeightsWarps) {
      const int key0 = u * kKv4Unit;
      auto& st = sm.stage[odd][warp];
      const uint32_t here = stage0 + odd * kStageBytes;
      cp_async_wait<0>();
      kv4_put_scales<D, false, false>(st, ks, ks, lane);
      __syncwarp();
      odd ^= 1;
      fetch(u + kKv4WeightsWarps, stage0 + odd * kStageBytes);
      const bool masked = key0 + kKv4Unit > all_see;
      const int key = key0 + g + 8 * t;   // the lane's weight
      float* weight = p.weights + bh * p.cap + key;
      const float old = key < len ? *weight : 0.0f;
      float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};   // keys g + 8 i
#pragma unroll
      for (int half0 = 0; half0 < 2; half0 += kSide) {
        uint32_t ka[kSide][D / 32], kb[kSide][D / 32];
        float sa[kSide][D / 32], sb[kSide][D / 32];
#pragma unroll
        for (int n = 0; n < kSide; ++n) {
          kv4_take_keys<D>(ka[n], kb[n], here + kv4_key_place<D>(lane), half0 + n);
          kv4_take_scales<D>(sa[n], &st.ks[(16 * (half0 + n) + g) * (D / 32)]);
          kv4_take_scales<D>(sb[n], &st.ks[(16 * (half0 + n) + 8 + g) * (D / 32)]);
        }
        for (int i = 0; i < p.rows; i += 8) {
          const auto& q = sm.q[i / 8];
          float s[kSide][4];
#pragma unroll
          for (int w = 0; w < D / 32; ++w) {
            const uint4 qb = q.b[w][lane];
            const float2 init = q.init[w][lane];
#pragma unroll
            for (int n = 0; n < kSide; ++n)
              kv4_score_group(s[n], w, ka[n][w], kb[n][w], sa[n][w], sb[n][w], qb, init);
          }
          const float2 factor = q.factor[lane], ref = *reinterpret_cast<const float2*>(&sm.ref[i + 2 * t]);
#pragma unroll
          for (int n = 0; n < kSide; ++n) {
            float e[4] = {ex2_approx(fmaf(s[n][0], factor.x, -ref.x)), ex2_approx(fmaf(s[n][1], factor.y, -ref.y)),
                          ex2_approx(fmaf(s[n][2], factor.x, -ref.x)), ex2_approx(fmaf(s[n][3], factor.y, -ref.y))};
            if (masked) {
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const int lim = sm.limit[i + 2 * t + c] - key0 - 16 * (half0 + n) - g;
                if (lim <= 0) e[c] = 0.0f;
                if (lim <= 8) e[2 + c] = 0.0f;
              }
            }
            sum[2 * (half0 + n)] += e[0] + e[1];
            sum[2 * (half0 + n) + 1] += e[2] + e[3];
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], 1);
        sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], 2);
      }
      const float mine = t == 0 ? sum[0] : t == 1 ? sum[1] : t == 2 ? sum[2] : sum[3];
      if (key < len) *weight = old + mine;
    }
    if (todo <= 0) return;
    r0 = -kKv4SegmentStart;
    if (++h == p.Hkv) {
      h = 0;
      do {
        len = p.length(++b);
        n_units = kv4_units(len);
      } while (n_units == 0);
    }
    __syncthreads();   // queries, references and limits are the next head's
  }
}

}  // namespace pasa
