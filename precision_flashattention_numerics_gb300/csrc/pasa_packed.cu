// libpasa.so: the C ABI of rotary positions and of attention over packed prompts (include/pasa.h).
#include <algorithm>
#include <cmath>

#include "host_util.cuh"
#include "packed_fwd.cuh"
#include "rope.cuh"

namespace {

int type_size(int type) { return type == PASA_TYPE_F32 ? 4 : type == PASA_TYPE_F16 || type == PASA_TYPE_BF16 ? 2 : 0; }

// Whether every row starts on a 16-byte boundary.
bool rows16(const void* p, const long long* strides, int size) {
  const long long step = 16 / size;
  return aligned16(p) && strides[0] % step == 0 && strides[1] % step == 0 && strides[2] % step == 0;
}

template <typename TIn, typename TOut>
void rope_launch(const pasa::RopeParams& p, bool vectors, bool interleaved, unsigned grid, cudaStream_t st) {
  auto kern = vectors ? (interleaved ? pasa::rope_kernel<TIn, TOut, true> : pasa::rope_kernel<TIn, TOut, false>)
                      : (interleaved ? pasa::rope_pairs_kernel<TIn, TOut, true> : pasa::rope_pairs_kernel<TIn, TOut, false>);
  kern<<<grid, pasa::kRopeThreads, 0, st>>>(p);
}

using PackedParams = pasa::packed::Params;

// The query heads of a tile: of the divisors of a kv head's g, the one whose tiles take the least time if every
// sequence has the mean length. A tile of d heads holds 128 / d tokens; long sequences want tiles without a spare row (g = 7:
// 18 x 7 rows of 128), short ones tiles that are not mostly empty. Equal ones: more heads, whose rows of a
// token lie side by side.
int packed_heads(int g, int N, int Tq) {
  const int mean = std::max(1, Tq / N);
  int best = 1;
  long long least = LLONG_MAX;
  for (int d = 1; d <= std::min(g, pasa::kTileRows); ++d) {
    if (g % d != 0) continue;
    const int tokens = pasa::kTileRows / d;
    const long long tiles = static_cast<long long>(g / d) * ((mean + tokens - 1) / tokens);
    if (tiles <= least) least = tiles, best = d;
  }
  return best;
}

struct PackedPlan {
  int hg, tile_tokens;
  long long tile_slots, key_slots;
  bool split;                           // whether tiles may be divided
  size_t tiles, splits, part_o, part_ml, kshift, means, total;   // workspace: byte offsets (the counts are at 0) and size
};

bool packed_fits(int N, int Hq, int Hkv, int Tq, int Tk) {
  if (N <= 0 || Hq <= 0 || Hkv <= 0 || Tq <= 0 || Tk <= 0 || Hq % Hkv != 0) return false;
  // row numbers past a last tile or block, and grids, fit an int
  if (Tq > INT_MAX - 512 || Tk > INT_MAX - 512 || N > INT_MAX - 512) return false;
  return (static_cast<long long>(Tq) + N) * Hq <= INT_MAX && (Tk / pasa::packed::kKeys + 1ll + N) * Hkv < INT_MAX;
}

PackedPlan packed_plan(int N, int Hq, int Hkv, int Tq, int Tk, int D, int mode) {
  PackedPlan pl = {};
  pl.hg = packed_heads(Hq / Hkv, N, Tq);
  pl.tile_tokens = pasa::kTileRows / pl.hg;
  pl.tile_slots = static_cast<long long>(Tq / pl.tile_tokens) + N;
  pl.key_slots = static_cast<long long>(Tk / pasa::packed::kKeys) + N;
  const bool shift = mode == PASA_MODE_SHIFT_F16ACC || mode == PASA_MODE_SHIFT_F32ACC;
  // Only where CTAs may be too few for the SMs, and keys enough for two pieces: then the list has room for all pieces, and
  // a launch more joins them (3 us where there is nothing to be joined).
  const long long groups = Hq / pl.hg;
  constexpr int kMaxPieces = pasa::packed::kMaxPieces;
  pl.split = pl.tile_slots * groups < kMaxPieces && Tk >= 2 * pasa::packed::kMinPiece * pasa::packed::kKeys;
  const size_t parts = pl.split ? kMaxPieces : 0;   // of all groups
  const size_t list = std::max<size_t>(pl.tile_slots, parts);
  pl.tiles = 256;
  pl.splits = pl.tiles + align_up(list * sizeof(pasa::packed::Tile), 256);
  pl.part_o = pl.splits + align_up(parts / 2 * sizeof(pasa::packed::Split), 256);
  pl.part_ml = pl.part_o + parts * pasa::kTileRows * D * 4;
  pl.kshift = pl.part_ml + parts * pasa::kTileRows * 8;
  pl.means = pl.kshift + (shift ? align_up(static_cast<size_t>(Hkv) * Tk * D * 2, 256) : 0);
  pl.total = pl.means + (shift ? align_up(static_cast<size_t>(Hkv) * pl.key_slots * D * 2, 256) : 0);
  return pl;
}

template <int D, bool F16ACC, bool SHIFT, bool PIECES>
int packed_launch(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mo,
                  const CUtensorMap& mm, const PackedParams& p, cudaStream_t st) {
  // ring slots as in pasa_attn_fwd: 3 K + 2 V for D = 128 (201 KB), 4 + 4 for D = 64
  constexpr int KST = D == 128 ? 3 : 4, VST = D == 128 ? 2 : 4;
  const unsigned prep = 1u + (SHIFT ? static_cast<unsigned>(p.key_slots) * static_cast<unsigned>(p.Hkv) : 0u);
  static std::atomic<unsigned long long> asked{0};
  prefer_shared(pasa::packed::packed_prep_kernel<D, PIECES>, asked);
  pasa::packed::packed_prep_kernel<D, PIECES><<<prep, pasa::packed::kPrepThreads, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e);
  constexpr int SETS = D == 64 ? 2 : 1;
  auto kern = pasa::packed::packed_fwd_kernel<D, F16ACC, SHIFT, KST, VST, SETS, PIECES>;
  const int smem = static_cast<int>(sizeof(pasa::packed::Smem<D, KST, VST, SETS>)) + 1024;
  static std::atomic<unsigned long long> raised{0};
  const unsigned groups = static_cast<unsigned>(p.Hq / p.hg);
  const unsigned most = std::max(static_cast<unsigned>(p.tile_slots), PIECES ? pasa::packed::kMaxPieces / groups : 0u);
  e = launch_clusters(kern, most * groups, pasa::packed::threads(SETS), smem, smem, st, true, 1, raised, mq, mk, mv, mo, mm, p);
  if constexpr (PIECES) {
    static std::atomic<unsigned long long> merge_asked{0};
    prefer_shared(pasa::packed::packed_merge_kernel<D>, merge_asked);
    if (e == cudaSuccess)
      e = launch_kernel(pasa::packed::packed_merge_kernel<D>, dim3(pasa::packed::kMergeCtas), dim3(pasa::packed::kMergeThreads), 0, st, true, p);
  }
  return e == cudaSuccess ? launch_status() : cuda_fail(e);
}

template <int D, bool PIECES>
int packed_dispatch(int mode, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mo,
                    const CUtensorMap& mm, const PackedParams& p, cudaStream_t st) {
  switch (mode) {
    case PASA_MODE_SHIFT_F16ACC: return packed_launch<D, true, true, PIECES>(mq, mk, mv, mo, mm, p, st);
    case PASA_MODE_SHIFT_F32ACC: return packed_launch<D, false, true, PIECES>(mq, mk, mv, mo, mm, p, st);
    case PASA_MODE_NAIVE_F16ACC: return packed_launch<D, true, false, PIECES>(mq, mk, mv, mo, mm, p, st);
    case PASA_MODE_NOSHIFT_F32ACC: return packed_launch<D, false, false, PIECES>(mq, mk, mv, mo, mm, p, st);
    default: return PASA_ERR_UNSUPPORTED;
  }
}

// Whether every row of [T, H, D] starts on a 16-byte boundary, and rows and heads do not fold onto one another.
int packed_layout(const void* p, const long long* strides, int T, int H, int D) {
  if (!aligned16(p) || strides[0] % 8 != 0 || strides[1] % 8 != 0) return PASA_ERR_ALIGN;
  const long long s3[3] = {0, strides[1], strides[0]};
  if (strides[0] <= 0 || strides[1] <= 0 || !strides_fit(s3, 1, H, T, D)) return PASA_ERR_SHAPE;
  if (strides[0] >= (1ll << 38) || strides[1] * H >= (1ll << 38)) return PASA_ERR_SHAPE;   // of a TMA descriptor
  return PASA_OK;
}

Strided packed_view(const void* p, const long long* strides, int T, int H, int D) {
  const long long s3[3] = {0, strides[1], strides[0]};
  return Strided(p, s3, 1, H, T, D, 2);
}

}  // namespace

namespace pasa {
int packed_take_device_error(DeviceError* found) { return take_device_error(found); }
int packed_wait_selftest(cudaStream_t st) { return launch_wait_selftest(st, true); }
}  // namespace pasa

extern "C" {

int pasa_rope_frequencies(double* inv_freq, float* mscale, int rotary_dim, double base, int scaling, double factor,
                          double original_length, double low, double high) {
  if (!inv_freq) return PASA_ERR_NULLPTR;
  if (rotary_dim < 2 || rotary_dim > pasa::kRopeMaxD || rotary_dim % 2 != 0) return PASA_ERR_SHAPE;
  if (scaling < PASA_ROPE_PLAIN || scaling > PASA_ROPE_BY_PARTS) return PASA_ERR_UNSUPPORTED;
  if (!(base > 1.0) || !std::isfinite(base)) return PASA_ERR_SHAPE;
  if (scaling != PASA_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return PASA_ERR_SHAPE;
  if (scaling == PASA_ROPE_BASE && rotary_dim < 4) return PASA_ERR_SHAPE;
  if (scaling == PASA_ROPE_BY_PARTS &&
      (!(original_length > 0.0) || !std::isfinite(original_length) || !(low >= 0.0) || !(high > low) || !std::isfinite(high)))
    return PASA_ERR_SHAPE;
  const double R = rotary_dim;
  if (scaling == PASA_ROPE_BASE) base *= std::pow(factor, R / (R - 2.0));
  for (int i = 0; i < rotary_dim / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / R);
    double x = f;
    if (scaling == PASA_ROPE_LINEAR) x = f / factor;
    if (scaling == PASA_ROPE_BY_PARTS) {
      const double turns = original_length * f / 6.283185307179586477;
      const double keep = std::fmin(1.0, std::fmax(0.0, (turns - low) / (high - low)));
      x = (1.0 - keep) * f / factor + keep * f;
    }
    inv_freq[i] = x;
  }
  if (mscale) *mscale = scaling == PASA_ROPE_BY_PARTS ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
  return PASA_OK;
}

int pasa_rope(const void* q, void* q_out, const long long* q_strides, int Hq, const void* k, void* k_out,
              const long long* k_strides, int Hkv, const double* inv_freq, const int* positions, const int* starts,
              int start, int B, int S, int D, int rotary_dim, int interleaved, int inverse, float mscale, int in_type,
              int out_type, void* stream) {
  if (!q || !q_out || !q_strides || !inv_freq) return PASA_ERR_NULLPTR;
  if (B <= 0 || S <= 0 || Hq <= 0 || Hkv < 0) return PASA_ERR_SHAPE;
  if (Hkv > 0 && (!k || !k_out || !k_strides)) return PASA_ERR_NULLPTR;
  if (D < 2 || D > pasa::kRopeMaxD || D % 2 != 0 || rotary_dim < 2 || rotary_dim > D || rotary_dim % 2 != 0) return PASA_ERR_SHAPE;
  if (!std::isfinite(mscale)) return PASA_ERR_SHAPE;
  const int in_size = type_size(in_type), out_size = type_size(out_type);
  if (in_size == 0 || out_size == 0 || (out_type != in_type && out_type != PASA_TYPE_F16)) return PASA_ERR_UNSUPPORTED;
  const long long heads = static_cast<long long>(Hq) + Hkv, tokens = static_cast<long long>(B) * S;
  if (heads > INT_MAX || tokens > INT_MAX) return PASA_ERR_SHAPE;
  const uintptr_t in_mask = in_size - 1, out_mask = out_size - 1;
  const void* ins[2] = {q, k};
  void* outs[2] = {q_out, k_out};
  const long long* strides[2] = {q_strides, k_strides};
  const int H[2] = {Hq, Hkv}, tensors = Hkv > 0 ? 2 : 1;
  bool vectors = rotary_dim % 16 == 0 && D % 8 == 0 && heads <= INT_MAX - 1024, in_place = true;   // (a head past the last fits an int)
  pasa::RopeParams p = {};
  for (int i = 0; i < tensors; ++i) {
    if ((reinterpret_cast<uintptr_t>(ins[i]) & in_mask) != 0 || (reinterpret_cast<uintptr_t>(outs[i]) & out_mask) != 0)
      return PASA_ERR_ALIGN;
    if (!strides_fit(strides[i], B, H[i], S, D) || !strides_fit(strides[i] + 3, B, H[i], S, D)) return PASA_ERR_SHAPE;
    vectors = vectors && rows16(ins[i], strides[i], in_size) && rows16(outs[i], strides[i] + 3, out_size);
    p.t[i] = pasa::RopeTensor{ins[i], outs[i], strides[i][0], strides[i][1], strides[i][2], strides[i][3], strides[i][4], strides[i][5]};
  }
  if ((reinterpret_cast<uintptr_t>(inv_freq) & 7u) != 0 || !aligned4(positions) || !aligned4(starts)) return PASA_ERR_ALIGN;
  // outputs: no row of one in another, and of the inputs only a tensor's own, element for element
  for (int i = 0; i < tensors; ++i) {
    const Strided out(outs[i], strides[i] + 3, B, H[i], S, D, out_size);
    if (out.folds()) return PASA_ERR_SHAPE;
    for (int j = 0; j < tensors; ++j) {
      const Strided in(ins[j], strides[j], B, H[j], S, D, in_size);
      if (i == j && in_type == out_type && out.same(in)) continue;
      if (out.meets(in)) return PASA_ERR_SHAPE;
      if (i == j) in_place = false;
      if (j < i && out.meets(Strided(outs[j], strides[j] + 3, B, H[j], S, D, out_size))) return PASA_ERR_SHAPE;
    }
    const Span o(outs[i], out.extent(0), 1);
    if (o.meets(Span(inv_freq, rotary_dim / 2, 8)) || o.meets(Span(positions, tokens, 4)) || o.meets(Span(starts, B, 4)))
      return PASA_ERR_SHAPE;
  }
  p.Hq = Hq;
  p.heads = static_cast<int>(heads);
  p.inv_freq = inv_freq;
  p.positions = positions;
  p.starts = starts;
  p.start = start;
  p.S = S;
  p.D = D;
  p.R = rotary_dim;
  p.mscale = mscale;
  p.sign = inverse ? -1.0f : 1.0f;
  long long ctas, part = tokens;   // tokens of a launch
  if (vectors) {
    p.groups = rotary_dim / 16 + (in_place ? 0 : (D - rotary_dim + 15) / 16);
    // head slots of a token: as few as fill the SMs, so that a thread's angles serve many heads, and a few times more where a
    // thread still has kRopeHeads heads (32768 tokens x 32 heads: 2 slots 106 us, 4 96, 8 98, 16 107)
    p.slots = 1;
    auto threads = [&] { return tokens * p.groups * p.slots; };
    while (p.slots < heads && (threads() < 152ll * 1024 || (threads() < 152ll * 4096 && 2ll * pasa::kRopeHeads * p.slots <= heads)))
      p.slots *= 2;
    p.slots = static_cast<unsigned>(std::min<long long>({p.slots, heads, static_cast<long long>(pasa::kRopeThreads / p.groups)}));
    p.cta_tokens = pasa::kRopeThreads / (p.groups * p.slots);
    ctas = (tokens + p.cta_tokens - 1) / p.cta_tokens;
  } else {
    p.groups = rotary_dim / 2 + (in_place ? 0 : D - rotary_dim);
    p.slots = static_cast<unsigned>(heads);
    const long long each = heads * p.groups;   // threads of a token
    part = std::min(tokens, (0xFFFFFF00ll - pasa::kRopeThreads) / each);
    if (part == 0) return PASA_ERR_SHAPE;
    ctas = (part * each + pasa::kRopeThreads - 1) / pasa::kRopeThreads;
  }
  const int rc = check_device();
  if (rc != PASA_OK) return rc;
  const unsigned grid = static_cast<unsigned>(ctas);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool same = in_type == out_type;
  for (long long first = 0; first < tokens; first += part) {
    p.token0 = static_cast<unsigned>(first);
    p.tokens = static_cast<unsigned>(std::min(tokens, first + part));
    if (in_type == PASA_TYPE_F16) rope_launch<__half, __half>(p, vectors, interleaved, grid, st);
    else if (in_type == PASA_TYPE_BF16 && same) rope_launch<__nv_bfloat16, __nv_bfloat16>(p, vectors, interleaved, grid, st);
    else if (in_type == PASA_TYPE_BF16) rope_launch<__nv_bfloat16, __half>(p, vectors, interleaved, grid, st);
    else if (same) rope_launch<float, float>(p, vectors, interleaved, grid, st);
    else rope_launch<float, __half>(p, vectors, interleaved, grid, st);
  }
  return launch_status();
}

size_t pasa_attn_fwd_packed_workspace_bytes(int N, int Hq, int Hkv, int Tq, int Tk, int D, int mode) {
  if (!packed_fits(N, Hq, Hkv, Tq, Tk) || (D != 64 && D != 128)) return 0;
  if (mode < PASA_MODE_SHIFT_F16ACC || mode > PASA_MODE_NOSHIFT_F32ACC) return 0;
  return packed_plan(N, Hq, Hkv, Tq, Tk, D, mode).total;
}

int pasa_attn_fwd_packed(const void* q, const void* k, const void* v, void* o, const long long* strides, float* lse,
                         const int* cu_q, const int* cu_k, int N, int Hq, int Hkv, int Tq, int Tk, int D, int causal,
                         float scale, int mode, void* workspace, size_t workspace_bytes, void* stream) {
  if (!q || !k || !v || !o || !strides || !cu_q || !cu_k) return PASA_ERR_NULLPTR;
  if (!packed_fits(N, Hq, Hkv, Tq, Tk)) return PASA_ERR_SHAPE;
  if ((D != 64 && D != 128) || mode < PASA_MODE_SHIFT_F16ACC || mode > PASA_MODE_NOSHIFT_F32ACC) return PASA_ERR_UNSUPPORTED;
  int rc;
  if ((rc = packed_layout(q, strides, Tq, Hq, D)) != PASA_OK || (rc = packed_layout(k, strides + 2, Tk, Hkv, D)) != PASA_OK ||
      (rc = packed_layout(v, strides + 4, Tk, Hkv, D)) != PASA_OK || (rc = packed_layout(o, strides + 6, Tq, Hq, D)) != PASA_OK)
    return rc;
  if (!aligned4(lse) || !aligned4(cu_q) || !aligned4(cu_k)) return PASA_ERR_ALIGN;
  const PackedPlan pl = packed_plan(N, Hq, Hkv, Tq, Tk, D, mode);
  if (!workspace || workspace_bytes < pl.total) return PASA_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return PASA_ERR_ALIGN;
  // o may be q itself: a CTA reads the rows that it writes, and no other CTA's result depends on them
  const Strided qs = packed_view(q, strides, Tq, Hq, D), ks = packed_view(k, strides + 2, Tk, Hkv, D);
  const Strided vs = packed_view(v, strides + 4, Tk, Hkv, D), os = packed_view(o, strides + 6, Tq, Hq, D);
  if (os.folds() || os.meets(ks) || os.meets(vs) || (os.meets(qs) && !os.same(qs))) return PASA_ERR_SHAPE;
  const Span out(o, os.extent(0), 1), ls(lse, static_cast<unsigned long long>(Hq) * Tq, 4), work(workspace, pl.total, 1);
  const Span cq(cu_q, N + 1ull, 4), ck(cu_k, N + 1ull, 4);
  if (any_meet({ls, work}, {out, Span(q, qs.extent(0), 1), Span(k, ks.extent(0), 1), Span(v, vs.extent(0), 1), cq, ck}) ||
      out.meets(cq) || out.meets(ck))
    return PASA_ERR_SHAPE;
  rc = check_device();
  if (rc != PASA_OK) return rc;
  if (!(scale > 0.0f) || !std::isfinite(scale)) scale = 1.0f / std::sqrt(static_cast<float>(D));
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  PackedParams p = {};
  p.cu_q = cu_q;
  p.cu_k = cu_k;
  p.N = N;
  p.Tq = Tq;
  p.Tk = Tk;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.hg = pl.hg;
  p.tile_tokens = pl.tile_tokens;
  int bits = 0;   // of tile_tokens - 1
  while ((1 << bits) < pl.tile_tokens) ++bits;
  p.tile_mul = static_cast<uint32_t>((((1ull << bits) - pl.tile_tokens) << 32) / pl.tile_tokens + 1);
  p.tile_shift1 = bits > 0 ? 1 : 0;
  p.tile_shift2 = bits > 0 ? bits - 1 : 0;
  p.tile_slots = static_cast<int>(pl.tile_slots);
  p.key_slots = static_cast<int>(pl.key_slots);
  p.causal = causal ? 1 : 0;
  while ((Tk / pasa::packed::kKeys + 1) >> p.bin_shift >= pasa::packed::kBins) ++p.bin_shift;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.inv_scale_log2 = 1.0f / p.scale_log2;
  p.count = reinterpret_cast<int*>(ws);
  p.tiles = reinterpret_cast<pasa::packed::Tile*>(ws + pl.tiles);
  p.splits = reinterpret_cast<pasa::packed::Split*>(ws + pl.splits);
  p.part_o = reinterpret_cast<float*>(ws + pl.part_o);
  p.part_ml = reinterpret_cast<float2*>(ws + pl.part_ml);
  p.k = static_cast<const __half*>(k);
  p.k_row = strides[2];
  p.k_head = strides[3];
  p.kshift = reinterpret_cast<__half*>(ws + pl.kshift);
  p.means = reinterpret_cast<__half*>(ws + pl.means);
  p.o = static_cast<__half*>(o);
  p.o_row = strides[6];
  p.o_head = strides[7];
  p.lse = lse;
  const bool shift = mode == PASA_MODE_SHIFT_F16ACC || mode == PASA_MODE_SHIFT_F32ACC;
  CUtensorMap mq, mk, mv, mo, mm;
  // (channels, heads of a tile, tokens, tiles' groups of heads) of q and o; (channels, rows, heads) of keys and values
  auto rows_map = [&](CUtensorMap* m, const void* at, const long long* s) {
    return make_strided_map(m, at, {D, pl.hg, Tq, Hq / pl.hg}, {s[1] * 2, s[0] * 2, s[1] * 2 * pl.hg}, {64, pl.hg, pl.tile_tokens, 1});
  };
  auto keys_map = [&](CUtensorMap* m, const void* at, long long row, long long head) {
    return make_strided_map(m, at, {D, Tk, Hkv}, {row * 2, head * 2}, {64, pasa::packed::kKeys, 1});
  };
  if ((rc = rows_map(&mq, q, strides)) != PASA_OK || (rc = rows_map(&mo, o, strides + 6)) != PASA_OK) return rc;
  if ((rc = shift ? keys_map(&mk, p.kshift, D, static_cast<long long>(Tk) * D) : keys_map(&mk, k, strides[2], strides[3])) != PASA_OK)
    return rc;
  if ((rc = keys_map(&mv, v, strides[4], strides[5])) != PASA_OK) return rc;
  mm = mk;   // unused without the shift
  if (shift && (rc = make_strided_map(&mm, p.means, {D, pl.key_slots, Hkv}, {D * 2, pl.key_slots * D * 2},
                                      {64, pasa::kChunkBlocks, 1})) != PASA_OK)
    return rc;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const auto run = D == 64 ? (pl.split ? packed_dispatch<64, true> : packed_dispatch<64, false>)
                           : (pl.split ? packed_dispatch<128, true> : packed_dispatch<128, false>);
  return run(mode, mq, mk, mv, mo, mm, p, st);
}

}  // extern "C"
