// Attention over packed sequences: token-major tensors [T, H, D] in which sequence s has the query rows
// cu_q[s] .. cu_q[s + 1] and the key rows cu_k[s] .. cu_k[s + 1], all lengths on the device.
//
// Method as in attn_fwd_kernel ("Online Pseudo-average Shifting Attention (PASA) for Robust Low-precision
// LLM Inference", arXiv 2503.01873, Abstract): every 128-key block of a sequence, counted from
// its first key, is shifted by its pseudo-average, scores are accumulated in fp16 or fp32, the offsets q_i . m_j
// are added back in fp32 in the online softmax.
//
// Two kernels. packed_prep_kernel shifts the keys (K' [Hkv, Tk, D], means [Hkv, slots, D]), and its first CTA
// writes the list of query tiles, those with the most key blocks first, so that uneven lengths leave
// no SM waiting at the end. packed_fwd_kernel takes a tile and a group of heads in each CTA.
//
// Tiles. A tile is 128 rows: `hg` query heads of one kv head (a divisor of Hq / Hkv) for each of 128 / hg tokens,
// row r token r / hg and head r mod hg, which one TMA box brings. Several heads to a tile fill
// the tiles of short sequences, where one head would leave most rows of its tile empty.
//
// Slots. Lengths are not known on the host, so key blocks get numbers that need no prefix sum: block j of
// sequence s is slot cu_k[s] / 128 + s + j. Those are distinct (a sequence of L keys from row c on has ceil(L / 128) blocks
// and floor((c + L) / 128) - floor(c / 128) + 1 slots to itself), and the sequence of a slot is found by a
// search in cu_k. Query tiles are numbered likewise.
//
// Pieces. Where a tile has more key blocks than an even share of all work (a chunk of a prompt on a long context, one
// long prompt with few heads), its blocks are divided among several CTAs, which leave partial results (O, max, sum)
// that packed_merge_kernel joins. piece_blocks() decides from the lengths, on the device. Measured with and without (mode 1,
// D = 128): 64 queries on 100000 keys, 32 heads on 8, 173 against 700 us; 128 on 20000, 1 on 8000 and 1 on 300, 28 on 4, 76
// against 186; a prompt of 16384, one head, 92 against 109. What is not divided pays the launch that finds nothing to join: 107
// against 104.5 us for four chunks. Kernels with and without PIECES are apart, as the little that it adds cost every
// call 2 us.
//
// Where a sequence ends inside a 128-key block, the block's last rows are another sequence's. Their scores are
// masked like any other, and their values are set to zero in shared memory before the MMA reads them: a
// probability of 0 does not make an infinity or NaN harmless.
//
// Bound by a block's chain of softmax and MMAs, as attn_fwd_kernel and attn_fwd_2set_kernel are: 32K tokens in 8 prompts, 28 heads,
// D = 128 1.94 ms, 1369 TFLOP/s (0.72 of the measured peak) in a graph that is replayed now and then, 2.06 ms, 1290 TFLOP/s (0.68) in
// calls one after the other, where power bounds the clock; D = 64, 4 prompts of up to 9216, 5 heads 102.7 us, 670 TFLOP/s, with no pipe
// full (exponentials 33%, tensor 32%, issue 44%: the chain's latency and the CTAs' starts and ends); 20
// prompts of up to 200 tokens 24.6 us (the latency of 2.2 waves of CTAs of 5 us each).
//
// cu_q and cu_k are clamped to their tensors and every number from them to its buffer: offsets that do not
// grow give unspecified results, but no access out of bounds.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_fp16.h>

#include "attn_fwd.cuh"
#include "kshift.cuh"
#include "ptx.cuh"

namespace pasa {
namespace packed {

constexpr int kKeys = 128;          // keys of a block
constexpr int kPrepThreads = 128;
constexpr int kBins = 1024;         // of the tiles' sort by their key blocks

// Pieces and their partial results: at most kMaxPieces, and of kMinPiece key blocks at least where their number is chosen.
constexpr int kSms = 152;
constexpr int kWaves = 4, kMaxPieces = kWaves * kSms;   // of CTAs, one to an SM
constexpr int kMinPiece = 8;
constexpr int kMinDivided = 2 * kMinPiece;   // blocks of the least tile that is divided: no sequence of fewer depends on its batch
constexpr int kPieceStart = 4;   // key blocks that the start and end of a CTA cost
constexpr int kMergeThreads = 256, kMergeCtas = 2 * kSms;

// One query tile, or a piece of its keys: all that a CTA has to know.
struct __align__(16) Tile {
  int q0, tokens;   // first token row of q, and how many
  int k0, keys;     // first key row of the sequence, and its keys
  int limit;        // keys that the first token sees, before clamping; each further one sees `step` more
  int step;         // 1 with the causal mask, else 0
  int blocks;       // key blocks that the last token sees
  int slot;         // of the sequence's first key block
  int pieces;       // of the tile; with more than one,
  int part;         // the number of this one among all pieces
  int unused[2];
};
// A tile in pieces.
struct __align__(16) Split {
  int q0, tokens;
  int part, pieces;   // the first piece's number, and how many
};

struct Params {
  const int *cu_q, *cu_k;
  int N, Tq, Tk, Hq, Hkv;
  int hg, tile_tokens;     // heads and tokens of a tile
  uint32_t tile_mul, tile_shift1, tile_shift2;   // x / tile_tokens is a product and two shifts
  int tile_slots, key_slots;
  int causal, bin_shift;
  float scale_log2, inv_scale_log2;
  int* count;              // tiles and pieces in the list; tiles in pieces
  Tile* tiles;
  Split* splits;           // with PIECES only, like the partial results
  float* part_o;           // [pieces][groups of heads][D / 4][rows][4]
  float2* part_ml;         // [pieces][groups of heads][rows]: max (log2 units), sum
  const __half* k;         // the raw keys, for the shift
  long long k_row, k_head; // their strides
  __half *kshift, *means;  // [Hkv, Tk, D], [Hkv, key_slots, D]
  __half* o;
  long long o_row, o_head;
  float* lse;              // [Hq, Tq] or nullptr
};

__device__ __forceinline__ int offset(const int* cu, int s, int most) { return min(max(__ldg(cu + s), 0), most); }

// The last s < n with start(s) <= slot, of those from lo on, by a whole warp: it probes 32 places at a time.
template <typename Start>
__device__ __forceinline__ int find_sequence(int lo, int hi, int slot, Start start) {
  const int lane = threadIdx.x & 31;
  while (hi - lo > 1) {   // the answer is in [lo, hi)
    const int step = (hi - lo + 31) / 32;
    const int s = lo + lane * step;
    const bool before = s < hi && start(s) <= slot;
    const uint32_t v = __ballot_sync(0xFFFFFFFFu, before) | 1u;   // lane 0: lo, by the loop's invariant
    const int last = 31 - __clz(v);
    lo += last * step;
    hi = min(hi, lo + step);
  }
  return lo;
}
// The number of a sequence's first tile.
__device__ __forceinline__ int first_tile(const Params& p, int s) {
  const uint32_t x = offset(p.cu_q, s, p.Tq), t = __umulhi(x, p.tile_mul);
  return static_cast<int>((t + ((x - t) >> p.tile_shift1)) >> p.tile_shift2) + s;   // x / tile_tokens + s
}
// The sequences of 32 slots side by side, slot0 + lane: the one of the first by search from lo on, those of the others among
// its 31 next ones, as each has a slot or more.
__device__ __forceinline__ int find_sequences(const Params& p, int lo, int slot0, int& mine) {
  const int lane = threadIdx.x & 31;
  lo = find_sequence(lo, min(p.N, lo + kPrepThreads + 1), slot0, [&](int s) { return first_tile(p, s); });
  const int start = lo + lane < p.N ? first_tile(p, lo + lane) : INT_MAX;
  int at = 0;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
    if (__shfl_sync(0xFFFFFFFFu, start, at + d) <= slot0 + lane) at += d;
  mine = lo + at;
  return lo;
}

// The tile of a slot; false where there is none.
__device__ __forceinline__ bool make_tile(const Params& p, int slot, int s, Tile& t) {
  if (slot >= p.tile_slots) return false;
  const int q0 = offset(p.cu_q, s, p.Tq), n = offset(p.cu_q, s + 1, p.Tq) - q0;
  const long long first = static_cast<long long>(slot - first_tile(p, s)) * p.tile_tokens;
  if (first < 0 || first >= n) return false;
  const int k0 = offset(p.cu_k, s, p.Tk), m = max(0, offset(p.cu_k, s + 1, p.Tk) - k0);
  const int i0 = static_cast<int>(first);
  t.q0 = q0 + i0;
  t.tokens = min(p.tile_tokens, n - i0);
  t.k0 = k0;
  t.keys = m;
  t.limit = p.causal ? i0 + 1 + m - n : m;
  t.step = p.causal ? 1 : 0;
  const int last = min(m, max(0, t.limit + t.step * (t.tokens - 1)));
  t.blocks = (last + kKeys - 1) / kKeys;
  t.slot = min(k0 / kKeys + s, p.key_slots - 1);
  t.pieces = 1;
  t.part = 0;
  return true;
}

// How many pieces a tile of so many key blocks is in, of `cap` blocks each at most.
__device__ __forceinline__ int pieces_of(int blocks, int cap) { return blocks < kMinDivided ? 1 : (blocks + cap - 1) / cap; }

// The most key blocks of a piece, or INT_MAX where no tile is to be divided. `sum`, `longest` and `tiles` of all tiles' blocks, and
// the longest of those that are too short to be divided, for each
// group of heads. Pieces of c blocks at most are no more than tiles + sum / c, so w waves of CTAs hold them with
// c = sum / (w SMs / groups - tiles), and take no longer than w (c + start), or the longest that is not divided, and the join. Undivided,
// the call takes longest + start at least: tiles are only divided where that is more, so that it always pays.
__device__ __forceinline__ int piece_blocks(const Params& p, long long sum, int longest, int longest_short, int tiles) {
  const int groups = p.Hq / p.hg;
  int best = INT_MAX;
  if (longest < kMinDivided) return best;
  long long least = (longest + kPieceStart) * 9ll / 10;   // by a tenth at least, for what the estimate leaves out
  for (int w = 1; w <= kWaves; ++w) {
    const int room = w * kSms / groups - tiles;
    if (room <= 0) continue;
    const long long c = max(static_cast<long long>(kMinPiece), (sum + room - 1) / room);
    const long long time = max(w * (c + kPieceStart), static_cast<long long>(longest_short + kPieceStart)) + 5 + longest / c / 5;
    if (c < longest && time < least) least = time, best = static_cast<int>(c);
  }
  return best;
}

// The list of tiles and pieces, most key blocks first: a counting sort by one CTA. Those of one bin come in any order, which
// no result depends on.
template <bool PIECES>
__device__ __forceinline__ void plan_tiles(const Params& p) {
  constexpr int kWarps = kPrepThreads / 32;
  __shared__ int bins[kBins];
  __shared__ int warp_sums[kWarps], warp_tiles[kWarps], warp_most[kWarps], warp_short[kWarps];
  __shared__ long long warp_blocks[kWarps];
  __shared__ int parts, splits;
  const int tid = threadIdx.x, lane = tid & 31;
  for (int i = tid; i < kBins; i += kPrepThreads) bins[i] = 0;
  if (tid == 0) parts = splits = 0;
  __syncthreads();
  // a thread keeps what it finds of its first few slots for the later passes
  constexpr int kKeep = 2;
  Tile kept[kKeep];
  bool there[kKeep];
  auto bin_of = [&](int blocks) { return kBins - 1 - min(kBins - 1, blocks >> p.bin_shift); };
  int tiles = 0, most = 0, most_short = 0;   // the longest tile, and of those that are not divided
  long long blocks = 0;
  auto count = [&](const Tile& t) {
    atomicAdd(&bins[bin_of(t.blocks)], 1);
    if (PIECES) {
      ++tiles, most = max(most, t.blocks), blocks += t.blocks;
      if (t.blocks < kMinDivided) most_short = max(most_short, t.blocks);
    }
  };
  const int tid0 = tid - lane;
  int lo = find_sequence(0, p.N, min(tid0, p.tile_slots - 1), [&](int s) { return first_tile(p, s); });
  const int lo0 = lo;
  int seq;
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {
    lo = find_sequences(p, lo, i * kPrepThreads + tid0, seq);
    there[i] = make_tile(p, i * kPrepThreads + tid, seq, kept[i]);
    if (there[i]) count(kept[i]);
  }
  const int lo1 = lo;
#pragma unroll 1
  for (int slot0 = kKeep * kPrepThreads + tid0; slot0 < p.tile_slots; slot0 += kPrepThreads) {
    Tile t;
    lo = find_sequences(p, lo, slot0, seq);
    if (make_tile(p, slot0 + lane, seq, t)) count(t);
  }
  __syncthreads();
  int cap = INT_MAX;
  if constexpr (PIECES) {
    tiles = __reduce_add_sync(0xFFFFFFFFu, tiles);
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    most_short = __reduce_max_sync(0xFFFFFFFFu, most_short);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) blocks += __shfl_xor_sync(0xFFFFFFFFu, blocks, d);
    if (lane == 0) {
      warp_tiles[tid >> 5] = tiles, warp_blocks[tid >> 5] = blocks;
      warp_most[tid >> 5] = most, warp_short[tid >> 5] = most_short;
    }
    __syncthreads();
    tiles = most = most_short = 0, blocks = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      tiles += warp_tiles[w], blocks += warp_blocks[w];
      most = max(most, warp_most[w]), most_short = max(most_short, warp_short[w]);
    }
    cap = piece_blocks(p, blocks, most, most_short, tiles);
    if (cap != INT_MAX) {   // count again
      for (int i = tid; i < kBins; i += kPrepThreads) bins[i] = 0;
      __syncthreads();
      lo = lo0;
#pragma unroll 1
      for (int slot0 = tid0; slot0 < p.tile_slots; slot0 += kPrepThreads) {
        Tile t;
        lo = find_sequences(p, lo, slot0, seq);
        if (!make_tile(p, slot0 + lane, seq, t)) continue;
        const int n = pieces_of(t.blocks, cap), base = t.blocks / n, more = t.blocks % n;
        atomicAdd(&bins[bin_of(base)], n - more);
        if (more > 0) atomicAdd(&bins[bin_of(base + 1)], more);
      }
      __syncthreads();
    }
  }
  // exclusive sums over the bins: 8 neighbouring ones a thread
  constexpr int kPer = kBins / kPrepThreads;
  int sum = 0, mine[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) mine[i] = bins[tid * kPer + i], sum += mine[i];
  int upto = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(0xFFFFFFFFu, upto, d);
    if (lane >= d) upto += x;
  }
  if (lane == 31) warp_sums[tid >> 5] = upto;
  __syncthreads();
  int before = upto - sum, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < (tid >> 5)) before += warp_sums[w];
    total += warp_sums[w];
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    bins[tid * kPer + i] = before;
    before += mine[i];
  }
  if (tid == 0) p.count[0] = total;
  __syncthreads();
  if (!PIECES || cap == INT_MAX) {
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
      if (there[i]) p.tiles[atomicAdd(&bins[bin_of(kept[i].blocks)], 1)] = kept[i];
    lo = lo1;
#pragma unroll 1
    for (int slot0 = kKeep * kPrepThreads + tid0; slot0 < p.tile_slots; slot0 += kPrepThreads) {
      Tile t;
      lo = find_sequences(p, lo, slot0, seq);
      if (make_tile(p, slot0 + lane, seq, t)) p.tiles[atomicAdd(&bins[bin_of(t.blocks)], 1)] = t;
    }
    if (PIECES && tid == 0) p.count[1] = 0;
    return;
  }
  if constexpr (PIECES) {
    lo = lo0;
#pragma unroll 1
    for (int slot0 = tid0; slot0 < p.tile_slots; slot0 += kPrepThreads) {
      Tile t;
      lo = find_sequences(p, lo, slot0, seq);
      if (!make_tile(p, slot0 + lane, seq, t)) continue;
      const int n = pieces_of(t.blocks, cap), base = t.blocks / n, more = t.blocks % n;
      t.pieces = n;
      if (n > 1) {
        t.part = atomicAdd(&parts, n);
        p.splits[atomicAdd(&splits, 1)] = Split{t.q0, t.tokens, t.part, n};
      }
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        t.blocks = base + (i < more ? 1 : 0);
        p.tiles[atomicAdd(&bins[bin_of(t.blocks)], 1)] = t;
        t.k0 += t.blocks * kKeys;
        t.keys -= t.blocks * kKeys;
        t.limit -= t.blocks * kKeys;
        t.slot += t.blocks;
        ++t.part;
      }
    }
    __syncthreads();
    if (tid == 0) p.count[1] = splits;
  }
}

// CTA 0 plans; CTA 1 + slot * Hkv + head shifts the key block of a slot (kshift_reg_kernel's arithmetic, bit for
// bit, on rows k_row apart). HBM-bound: each key is read once and written once.
template <int D, bool PIECES>
__global__ void __launch_bounds__(kPrepThreads) packed_prep_kernel(const __grid_constant__ Params p) {
  griddep_launch_dependents();
  if (blockIdx.x == 0) {
    plan_tiles<PIECES>(p);
    return;
  }
  const int slot = (blockIdx.x - 1) / p.Hkv, head = (blockIdx.x - 1) % p.Hkv;
  const int s = find_sequence(0, p.N, slot, [&](int i) { return offset(p.cu_k, i, p.Tk) / kKeys + i; });
  const int k0 = offset(p.cu_k, s, p.Tk), m = offset(p.cu_k, s + 1, p.Tk) - k0;
  const long long first = static_cast<long long>(slot - (k0 / kKeys + s)) * kKeys;
  if (first < 0 || first >= m) return;
  const int row0 = k0 + static_cast<int>(first);
  const int n = min(kKeys, m - static_cast<int>(first));
  shift_block<D, kKeys>(reinterpret_cast<const uint4*>(p.k + row0 * p.k_row + head * p.k_head), p.k_row / 8,
                        reinterpret_cast<uint4*>(p.kshift + (static_cast<long long>(head) * p.Tk + row0) * D), D / 8,
                        reinterpret_cast<uint4*>(p.means + (static_cast<long long>(head) * p.key_slots + slot) * D), n);
}

// Shared memory: attn_fwd_kernel's and, for two softmax sets, what they exchange.
template <int D, int KST, int VST, int SETS>
struct Smem : AttnSmem<D, kKeys, KST, VST> {
  uint64_t pv_done[2];           // PV(j), by the parity of j: with two sets, one can come to its wait for PV(j) while PV(j - 1)
                                 // still runs, and one barrier's phase of PV(j - 2) would look like PV(j)'s
  uint64_t mx_full[4][SETS];     // [rows 32 q ..][set]: the set has published m of its block
  float m_of[SETS][kTileRows];   // the maximum that a row's last block was taken with
  float2 sums[SETS][kTileRows];  // in the end: a row's sum, and the maximum it is scaled to
  int2 piece;                    // the tile's pieces and this one's number: out of the registers until the end
};
__host__ __device__ constexpr int threads(int sets) { return (4 * sets + 3) * 32; }

// One CTA: a tile of the list, or with PIECES maybe a piece of one, and a group of hg heads. Warp roles, TMEM and barriers as in attn_fwd_kernel (SETS = 1) and
// attn_fwd_2set_kernel (SETS = 2, for D = 64, whose MMAs take half as long beside the same softmax): 4 warps of softmax and
// epilogue, one thread per row, for each set, which take the blocks in turn; then a warp for TMA, one for the score and
// offsets MMAs, one for PV. All waits are bounded (ptx.cuh).
template <int D, bool F16ACC, bool SHIFT, int KST, int VST, int SETS, bool PIECES>
__global__ void __launch_bounds__(threads(SETS), 1)
packed_fwd_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                  const __grid_constant__ CUtensorMap mapV, const __grid_constant__ CUtensorMap mapO,
                  const __grid_constant__ CUtensorMap mapM, const __grid_constant__ Params p) {
  constexpr int BN = kKeys;
  using Smem = packed::Smem<D, KST, VST, SETS>;
  constexpr int kTma = 4 * SETS, kQk = kTma + 1, kPv = kTma + 2;   // warps
  static_assert(sizeof(Smem) + 1024 <= 227 * 1024, "shared memory per CTA");
  using TM = TmemMap<D, BN>;
  extern __shared__ uint8_t smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;

  if (tid == 0) {
    mbar_init(&s.q_full, 1);
    for (int i = 0; i < KST; ++i) { mbar_init(&s.k_full[i], 1); mbar_init(&s.k_empty[i], 1); }
    for (int i = 0; i < VST; ++i) { mbar_init(&s.v_full[i], 1); mbar_init(&s.v_empty[i], 1); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.m_full[i], 1);
      mbar_init(&s.m_empty[i], 1);
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.s_free[i], 4);
    }
    mbar_init(&s.p_full, 4);
    for (int i = 0; i < 2; ++i) mbar_init(&s.pv_done[i], 1);
    for (int i = 0; i < 4 * SETS; ++i) mbar_init(&s.mx_full[i / SETS][i % SETS], 1);
    mbar_init(&s.o_full, 1);
    mbar_init(&s.drain[0], 1);
    mbar_init(&s.drain[1], 1);
    s.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kTma && lane == 0) {
    tma_prefetch_desc(&mapQ);
    tma_prefetch_desc(&mapK);
    tma_prefetch_desc(&mapV);
    tma_prefetch_desc(&mapO);
    if (SHIFT) tma_prefetch_desc(&mapM);
  }
  if (warp == kQk) {
    tmem_alloc(&s.tmem_base, 512);
    tmem_relinquish();
  }
  const int groups = p.Hq / p.hg;
  const int item = blockIdx.x / groups, group = blockIdx.x % groups;
  if (PIECES) griddep_launch_dependents();   // the join, which waits for all of this
  griddep_wait();   // the list, the shifted keys and the means; every CTA: a kernel behind this one waits for this one
  const bool there = item < __ldcg(p.count);
  Tile t = {};
  if (there) {
    const int4* rec = reinterpret_cast<const int4*>(p.tiles + item);
    const int4 a = __ldcg(rec), b = __ldcg(rec + 1);
    t = Tile{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (PIECES && tid == 0) s.piece = __ldcg(reinterpret_cast<const int2*>(rec + 2));
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  volatile int* abort_flag = &s.abort_flag;
  const int nblk = t.blocks;
  const int rows = p.hg * p.tile_tokens;
  const int hk = group / (p.Hq / p.Hkv / p.hg);

  if (!there) {
    // nothing to do but to give the TMEM back
  } else if (warp == kTma) {
    // ------------------------------------------------------------------ TMA producer
    if (lane == 0) {
      const uint32_t q_chunk = static_cast<uint32_t>(rows) * 128;
      mbar_arrive_expect_tx(&s.q_full, q_chunk * Smem::kChunks);
#pragma unroll
      for (int c = 0; c < Smem::kChunks; ++c) tma_load_4d(s.q + c * Smem::kQChunk, &mapQ, &s.q_full, c * 64, 0, t.q0, group);
      int k_issued = 0, v_issued = 0, m_issued = 0;
      auto load_k = [&](int j) -> bool {
        if (SHIFT && (j % kChunkBlocks) == 0) {
          const int ci = j / kChunkBlocks, slot = ci & 1;
          if (!mbar_wait(&s.m_empty[slot], ((ci >> 1) & 1) ^ 1, abort_flag, 0x1101)) return false;
          mbar_arrive_expect_tx(&s.m_full[slot], Smem::kMTile);
#pragma unroll
          for (int c = 0; c < Smem::kChunks; ++c)
            tma_load_3d(s.m[slot] + c * Smem::kMChunk, &mapM, &s.m_full[slot], c * 64, t.slot + j, hk);
          m_issued = ci + 1;
        }
        const int ks = j % KST;
        if (!mbar_wait(&s.k_empty[ks], ((j / KST) & 1) ^ 1, abort_flag, 0x1102)) return false;
        mbar_arrive_expect_tx(&s.k_full[ks], Smem::kKTile);
#pragma unroll
        for (int c = 0; c < Smem::kChunks; ++c)
          tma_load_3d(s.k[ks] + c * Smem::kKChunk, &mapK, &s.k_full[ks], c * 64, t.k0 + j * BN, hk);
        k_issued = j + 1;
        return true;
      };
      auto load_v = [&](int j) -> bool {
        const int vs = j % VST;
        if (!mbar_wait(&s.v_empty[vs], ((j / VST) & 1) ^ 1, abort_flag, 0x1103)) return false;
        mbar_arrive_expect_tx(&s.v_full[vs], Smem::kVTile);
#pragma unroll
        for (int c = 0; c < Smem::kChunks; ++c)
          tma_load_3d(s.v[vs] + c * Smem::kVChunk, &mapV, &s.v_full[vs], c * 64, t.k0 + j * BN, hk);
        v_issued = j + 1;
        return true;
      };
      bool pok = nblk == 0 || load_k(0);
      for (int j = 0; pok && j < nblk; ++j) {
        if (j + 1 < nblk && !load_k(j + 1)) break;
        if (!load_v(j)) break;
      }
      if (*abort_flag) {
        // Let every copy this warp issued land before the CTA's shared memory goes away.
        const uint64_t t0 = globaltimer_ns();
        auto drain = [&](uint64_t* bar, uint32_t parity) {
          while (!mbar_try_wait(bar, parity) && globaltimer_ns() - t0 < kWaitTimeoutNs) {
          }
        };
        drain(&s.q_full, 0);
        for (int j = max(0, k_issued - KST); j < k_issued; ++j) drain(&s.k_full[j % KST], (j / KST) & 1);
        for (int j = max(0, v_issued - VST); j < v_issued; ++j) drain(&s.v_full[j % VST], (j / VST) & 1);
        for (int ci = max(0, m_issued - 2); ci < m_issued; ++ci) drain(&s.m_full[ci & 1], (ci >> 1) & 1);
      }
    }
    __syncwarp();
  } else if (warp == kQk) {
    // ------------------------------------------------------------------ QK issuer (see attn_fwd_kernel)
    if (lane == 0) {
      constexpr uint32_t id_s = idesc_f16(kTileRows, BN, !F16ACC, false);
      constexpr uint32_t id_c = idesc_f16(kTileRows, kChunkBlocks, true, false);
      constexpr uint32_t hi_kmaj = sdesc_hi_sw128(1024);
      const uint32_t q_lo = sdesc_lo(smem_u32(s.q), 16);
      const uint32_t k_lo0 = sdesc_lo(smem_u32(s.k[0]), 16);
      const uint32_t m_lo0 = sdesc_lo(smem_u32(s.m[0]), 16);
      constexpr uint32_t kKStride = sizeof(s.k[0]) >> 4;
      constexpr uint32_t kMStride = sizeof(s.m[0]) >> 4;
      uint32_t qd[D / 16];
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) qd[kk] = q_lo + (((kk / 4) * Smem::kQChunk + (kk % 4) * 32) >> 4);
      bool ok = mbar_wait(&s.q_full, 0, abort_flag, 0x1201);
      const uint32_t tQ = tmem + TM::q;
      constexpr int kQt = TM::kQtSteps;
      if (ok && nblk > 0) {
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kQt; ++kk) tmem_cp_128x256b(tQ + kk * 8, qd[kk], hi_kmaj);
      }
      for (int j = 0; ok && j < nblk; ++j) {
        const int ks = j % KST;
        const int ci = j / kChunkBlocks;
        const int sb = j & 1;
        const bool chunk_start = SHIFT && (j % kChunkBlocks) == 0;
        uint32_t kd[D / 16];
        const uint32_t k_lo = k_lo0 + ks * kKStride;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) kd[kk] = k_lo + (((kk / 4) * Smem::kKChunk + (kk % 4) * 32) >> 4);
        if (!mbar_wait(&s.k_full[ks], (j / KST) & 1, abort_flag, 0x1202)) break;
        if (chunk_start && !mbar_wait(&s.m_full[ci & 1], (ci >> 1) & 1, abort_flag, 0x1203)) break;
        if (j >= 2 && !mbar_wait(&s.s_free[sb], ((j >> 1) - 1) & 1, abort_flag, 0x1206)) break;
        tc_fence_after();
        if (chunk_start) {
          const uint32_t m_lo = m_lo0 + (ci & 1) * kMStride;
          const uint32_t tC = tmem + TM::c(ci & 1);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off_m = ((kk / 4) * Smem::kMChunk + (kk % 4) * 32) >> 4;
            if (kk < kQt) mma_ts_w(tC, tQ + kk * 8, m_lo + off_m, hi_kmaj, id_c, kk > 0 ? 1u : 0u);
            else mma_ss_w(tC, qd[kk], hi_kmaj, m_lo + off_m, hi_kmaj, id_c, kk > 0 ? 1u : 0u);
          }
        }
        const uint32_t tS = tmem + TM::s(sb);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          if (kk < kQt) mma_ts_w(tS, tQ + kk * 8, kd[kk], hi_kmaj, id_s, kk > 0 ? 1u : 0u);
          else mma_ss_w(tS, qd[kk], hi_kmaj, kd[kk], hi_kmaj, id_s, kk > 0 ? 1u : 0u);
        }
        mma_commit(&s.s_full[sb]);
        mma_commit(&s.k_empty[ks]);
        if (chunk_start) mma_commit(&s.m_empty[ci & 1]);
      }
      mma_commit(&s.drain[0]);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(&s.drain[0], 0) && globaltimer_ns() - t0 < kWaitTimeoutNs) {
      }
    }
    __syncwarp();
  } else if (warp == kPv) {
    // ------------------------------------------------------------------ PV issuer
    if (lane == 0) {
      constexpr uint32_t id_o = idesc_f16(kTileRows, D, true, true);
      constexpr uint32_t hi_v = sdesc_hi_sw128(1024);
      const uint32_t v_lo0 = sdesc_lo(smem_u32(s.v[0]), Smem::kVChunk);
      constexpr uint32_t kVStride = sizeof(s.v[0]) >> 4;
      const uint32_t tO = tmem + TM::o;
      const uint32_t tP = tmem + TM::p;
      for (int j = 0; j < nblk; ++j) {
        const int vs = j % VST;
        uint32_t vd[BN / 16];
        const uint32_t v_lo = v_lo0 + vs * kVStride;
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk) vd[kk] = v_lo + kk * (2048 >> 4);
        if (!mbar_wait(&s.v_full[vs], (j / VST) & 1, abort_flag, 0x1204)) break;
        if (!mbar_wait(&s.p_full, j & 1, abort_flag, 0x1205)) break;
        tc_fence_after();
        const uint32_t acc0 = j > 0 ? 1u : 0u;
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk) mma_ts_w(tO, tP + kk * 8, vd[kk], hi_v, id_o, kk > 0 ? 1u : acc0);
        mma_commit(&s.pv_done[j & 1]);
        mma_commit(&s.v_empty[vs]);
        if (j == nblk - 1) mma_commit(&s.o_full);
      }
      mma_commit(&s.drain[1]);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(&s.drain[1], 0) && globaltimer_ns() - t0 < kWaitTimeoutNs) {
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ softmax + epilogue
    const int set = SETS == 1 ? 0 : warp >> 2, quad = warp & 3;
    const int r = quad * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t tO = tmem + lane_base + TM::o;
    const uint32_t tP = tmem + lane_base + TM::p;
    const int token = r / p.hg;
    const bool live = token < t.tokens;
    const int limit = live ? min(t.keys, max(0, t.limit + t.step * token)) : 0;
    const float sl2 = p.scale_log2;
    constexpr int kPairs = BN / 2;
    float m_run = -INFINITY, l_run = 0.0f;   // with two sets: this one's sum, and the maximum it is scaled to
    bool ok = true;
    // values of the last block that are not this sequence's (none past the tensor, where TMA fills with zeros)
    const int foreign = t.k0 + t.keys < p.Tk ? t.keys - (nblk - 1) * BN : BN;

    for (int j = set; ok && j < nblk; j += SETS) {
      const int sb = j & 1;
      if (!mbar_wait(&s.s_full[sb], (j >> 1) & 1, abort_flag, 0x1300)) { ok = false; break; }
      tc_fence_after();
      const uint32_t tS = tmem + lane_base + TM::s(sb);
      uint32_t hp[F16ACC ? kPairs : 1];
      float sv[F16ACC ? 1 : BN];
      uint32_t cw = 0;
      if constexpr (F16ACC) {
        tmem_ld_scores_f16<BN>(tS, hp);
      } else {
#pragma unroll
        for (int c = 0; c < BN / 16; ++c) tmem_ld_x16(tS + c * 16, reinterpret_cast<uint32_t*>(sv) + c * 16);
      }
      if (SHIFT) tmem_ld_x1(tmem + lane_base + TM::c((j / kChunkBlocks) & 1) + (j % kChunkBlocks), cw);
      tmem_ld_wait();
      if constexpr (F16ACC) reg_fence<kPairs>(hp);
      else reg_fence<BN>(reinterpret_cast<uint32_t*>(sv));
      reg_fence<1>(&cw);
      tc_fence_before();
      __syncwarp();
      mbar_arrive_if(&s.s_free[sb], lane == 0);

      const int cmax = limit - j * BN;
      const float c_raw = SHIFT ? __uint_as_float(cw) : 0.0f;
      float mx;
      if constexpr (F16ACC) {
        if (cmax < BN) {
#pragma unroll
          for (int c = 0; c < kPairs; ++c)
            hp[c] = ((2 * c < cmax) ? (hp[c] & 0xFFFFu) : 0xFC00u) |
                    ((2 * c + 1 < cmax) ? (hp[c] & 0xFFFF0000u) : 0xFC000000u);  // -inf when masked
        }
        uint32_t tmp[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) tmp[k] = hp[k];
#pragma unroll
        for (int c = 8; c < kPairs; ++c) tmp[c & 7] = hmax2(tmp[c & 7], hp[c]);
        const uint32_t m1 = tree_h2<8, true>(tmp);
        mx = fmaxf(half_lo_to_float(m1), half_lo_to_float(m1 >> 16));
      } else {
        if (cmax < BN) {
#pragma unroll
          for (int c = 0; c < BN; ++c)
            if (c >= cmax) sv[c] = -INFINITY;
        }
        float tmp[BN];
#pragma unroll
        for (int c = 0; c < BN; ++c) tmp[c] = sv[c];
        mx = tree_max3<BN>(tmp);
      }
      const float bm = (mx == -INFINITY) ? -INFINITY : (mx + c_raw) * sl2;
      float m_prev = m_run;   // what the block before was taken with
      if (SETS == 2 && j > 0) {
        if (!mbar_wait(&s.mx_full[quad][set ^ (SETS - 1)], ((j - 1) >> 1) & 1, abort_flag, 0x1340)) { ok = false; break; }
        m_prev = s.m_of[set ^ (SETS - 1)][r];
      }
      const float m_new = fmaxf(m_prev, bm);
      const bool need = m_new > m_prev + kRescaleLog2;
      const bool later = j > 0;
      const float alpha_n = ex2_approx(m_prev - m_new);
      const float alpha = need ? alpha_n : 1.0f;
      const float m_cur = (need || !later) ? m_new : m_prev;
      if constexpr (SETS == 2) {
        s.m_of[set][r] = m_cur;
        __syncwarp();
        mbar_arrive_if(&s.mx_full[quad][set], lane == 0);
        if (m_run != m_cur) l_run *= ex2_approx(m_run - m_cur);   // 0 while this set has no block yet
      } else {
        l_run = (need && later) ? l_run * alpha_n : l_run;
      }
      m_run = m_cur;
      const bool rescale = __any_sync(0xffffffffu, need) && later;
      float rs[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      uint32_t pk[kPairs];
      if constexpr (F16ACC) {
        const float b16 = (m_run == -INFINITY) ? 0.0f : c_raw - m_run * p.inv_scale_log2;
#pragma unroll
        for (int c = 0; c < kPairs; ++c) {
          float y0, y1, x0, x1;
          add_f16x2_f32(y0, y1, hp[c], b16);
          fmul2(x0, x1, y0, y1, sl2, sl2);
          const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
          pk[c] = pack_half2(p0, p1);
          const int a = (c & 3) * 2;
          fadd2(rs[a], rs[a + 1], rs[a], rs[a + 1], p0, p1);
        }
      } else {
        const float bias = (m_run == -INFINITY) ? 0.0f : c_raw * sl2 - m_run;
#pragma unroll
        for (int c = 0; c < kPairs; ++c) {
          float x0, x1;
          ffma2(x0, x1, sv[2 * c], sv[2 * c + 1], sl2, sl2, bias, bias);
          const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
          const int a = (c & 3) * 2;
          fadd2(rs[a], rs[a + 1], rs[a], rs[a + 1], p0, p1);
          pk[c] = pack_half2(p0, p1);
        }
      }
      l_run += ((rs[0] + rs[1]) + (rs[2] + rs[3])) + ((rs[4] + rs[5]) + (rs[6] + rs[7]));
      if (j >= 1 && !mbar_wait(&s.pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1, abort_flag, 0x1320)) { ok = false; break; }
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < BN / 16; ++c) tmem_st_x8(tP + c * 8, pk + c * 8);
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
      if (j == nblk - 1 && foreign < BN) {
        // thread r: the zeros of value row r (one 128-byte row of each 64-channel chunk)
        const int vs = j % VST;
        if (!mbar_wait(&s.v_full[vs], (j / VST) & 1, abort_flag, 0x1321)) { ok = false; break; }
        if (r >= foreign) {
#pragma unroll
          for (int c = 0; c < Smem::kChunks; ++c)
#pragma unroll
            for (int u = 0; u < 8; ++u)
              *reinterpret_cast<uint4*>(s.v[vs] + c * Smem::kVChunk + r * 128 + ((u ^ (r & 7)) * 16)) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
        }
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      mbar_arrive_if(&s.p_full, lane == 0);
    }

    // epilogue: O / l -> fp16 -> swizzled staging (the Q buffer) -> TMA store, or for a sequence's last tile, whose
    // box would run into the next sequence, row by row
    const bool have_o = ok && nblk > 0;
    if (have_o && !mbar_wait(&s.o_full, 0, abort_flag, 0x1310)) ok = false;
    if (!have_o && !mbar_wait(&s.q_full, 0, abort_flag, 0x1330)) ok = false;
    tc_fence_after();
    if constexpr (SETS == 2) {
      s.sums[set][r] = make_float2(l_run, m_run);
      named_bar_sync(1, 128 * SETS);
      const float2 other = s.sums[set ^ (SETS - 1)][r];
      const float m_f = fmaxf(m_run, other.y);   // what O is scaled to: the last block's
      // without a maximum both sums are 0, or NaN for a NaN query
      l_run = m_f == -INFINITY ? l_run + other.x : l_run * ex2_approx(m_run - m_f) + other.x * ex2_approx(other.y - m_f);
      m_run = m_f;
    }
    const int2 piece = PIECES ? s.piece : make_int2(1, 0);
    const bool part = piece.x > 1;
    const float inv_l = part ? 1.0f : l_run == 0.0f ? 0.0f : 1.0f / l_run;
    const long long at = static_cast<long long>(piece.y) * groups + group;   // of the partial results
    uint8_t* stage = s.q;
    constexpr int kCols = D / SETS;   // of O, for a set
#pragma unroll
    for (int c0 = 0; c0 < kCols; c0 += 32) {
      const int c = set * kCols + c0;
      uint32_t w[32];
      if (have_o && ok) {
        tmem_ld_x16(tO + c, w);
        tmem_ld_x16(tO + c + 16, w + 16);
        tmem_ld_wait();
        reg_fence<32>(w);
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) w[e] = 0u;
      }
      if (part) {
        float4* to = reinterpret_cast<float4*>(p.part_o) + (at * (D / 4) + c / 4) * kTileRows + r;
#pragma unroll
        for (int u = 0; u < 8; ++u)
          to[u * kTileRows] = make_float4(__uint_as_float(w[4 * u]), __uint_as_float(w[4 * u + 1]), __uint_as_float(w[4 * u + 2]),
                                          __uint_as_float(w[4 * u + 3]));
        continue;
      }
      uint8_t* rowp = stage + c / 64 * Smem::kQChunk + r * 128;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          h[e] = pack_half2(__uint_as_float(w[8 * u + 2 * e]) * inv_l, __uint_as_float(w[8 * u + 2 * e + 1]) * inv_l);
        *reinterpret_cast<uint4*>(rowp + (((c % 64 / 8 + u) ^ (r & 7)) * 16)) = make_uint4(h[0], h[1], h[2], h[3]);
      }
    }
    if (part && set == 0) p.part_ml[at * kTileRows + r] = make_float2(m_run, l_run);
    const bool whole = !part && t.tokens == p.tile_tokens;
    if (whole) fence_proxy_async_smem();
    named_bar_sync(2, 128 * SETS);
    if (whole) {
      if (tid == 0) {
#pragma unroll
        for (int c = 0; c < Smem::kChunks; ++c) tma_store_4d(&mapO, stage + c * Smem::kQChunk, c * 64, 0, t.q0, group);
        tma_store_commit();
        tma_store_wait_read();   // the stage stays until it has been read; the rows land in their own time
      }
    } else if (!part) {
      constexpr int kU = D / 8;   // 16-byte units of a row
      for (int e = tid; e < t.tokens * p.hg * kU; e += 128 * SETS) {
        const int row = e / kU, u = e % kU;
        const uint4 x = *reinterpret_cast<const uint4*>(stage + (u / 8) * Smem::kQChunk + row * 128 + (((u % 8) ^ (row & 7)) * 16));
        __half* to = p.o + (t.q0 + row / p.hg) * p.o_row + (group * p.hg + row % p.hg) * p.o_head + u * 8;
        *reinterpret_cast<uint4*>(to) = x;
      }
    }
    if (p.lse != nullptr && live && set == 0 && !part) {
      const float lse = l_run == 0.0f ? -INFINITY : (m_run + log2f(l_run)) * 0.69314718055994531f;
      p.lse[static_cast<long long>(group * p.hg + r % p.hg) * p.Tq + t.q0 + token] = lse;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kQk) tmem_dealloc(tmem, 512);
}

// Joins the pieces of tiles. A CTA takes 8 channels of a tile's rows and group of heads, a thread 4 of one row.
template <int D>
__global__ void __launch_bounds__(kMergeThreads, 4) packed_merge_kernel(const __grid_constant__ Params p) {
  static_assert(kMergeThreads == 2 * kTileRows, "two threads to a row");
  const int groups = p.Hq / p.hg;
  const int r = threadIdx.x % kTileRows;
  griddep_wait();
  const int todo = __ldcg(p.count + 1) * groups * (D / 8);
#pragma unroll 1
  for (int i = blockIdx.x; i < todo; i += gridDim.x) {
    const int ch = (i % (D / 8) * 2 + threadIdx.x / kTileRows) * 4;
    const int group = i / (D / 8) % groups;
    const int4 rec = __ldcg(reinterpret_cast<const int4*>(p.splits + i / (D / 8) / groups));
    const Split t = Split{rec.x, rec.y, rec.z, rec.w};
    const int token = r / p.hg;
    if (token >= t.tokens) continue;
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float m_run = -INFINITY, l_run = 0.0f;
    constexpr int kAtOnce = 4;
#pragma unroll 1
    for (int i0 = 0; i0 < t.pieces; i0 += kAtOnce) {
      float2 ml[kAtOnce];
      float4 v[kAtOnce];
#pragma unroll
      for (int e = 0; e < kAtOnce; ++e) {
        const long long at = static_cast<long long>(t.part + i0 + e) * groups + group;
        ml[e] = make_float2(-INFINITY, 0.0f);
        v[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (i0 + e < t.pieces) {
          ml[e] = __ldcg(p.part_ml + at * kTileRows + r);
          v[e] = __ldcg(reinterpret_cast<const float4*>(p.part_o) + (at * (D / 4) + ch / 4) * kTileRows + r);
        }
      }
      float top = m_run;
#pragma unroll
      for (int e = 0; e < kAtOnce; ++e) top = fmaxf(top, ml[e].x);
      if (top == -INFINITY) {   // pieces of which the row sees nothing, or of a NaN query, whose sums are NaN
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e) l_run += ml[e].y;
        continue;
      }
      const float f0 = ex2_approx(m_run - top);
      l_run *= f0, x.x *= f0, x.y *= f0, x.z *= f0, x.w *= f0;
      m_run = top;
#pragma unroll
      for (int e = 0; e < kAtOnce; ++e) {
        const float f = ex2_approx(ml[e].x - top);
        l_run = fmaf(f, ml[e].y, l_run);
        x.x = fmaf(f, v[e].x, x.x), x.y = fmaf(f, v[e].y, x.y), x.z = fmaf(f, v[e].z, x.z), x.w = fmaf(f, v[e].w, x.w);
      }
    }
    const float inv = l_run == 0.0f ? 0.0f : 1.0f / l_run;
    const int head = group * p.hg + r % p.hg;
    *reinterpret_cast<uint2*>(p.o + (t.q0 + token) * p.o_row + head * p.o_head + ch) =
        make_uint2(pack_half2(x.x * inv, x.y * inv), pack_half2(x.z * inv, x.w * inv));
    if (ch == 0 && p.lse)
      p.lse[static_cast<long long>(head) * p.Tq + t.q0 + token] = l_run == 0.0f ? -INFINITY : (m_run + log2f(l_run)) * 0.69314718055994531f;
  }
}

}  // namespace packed
}  // namespace pasa
