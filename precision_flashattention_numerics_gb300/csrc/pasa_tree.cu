// libpasa.so: the C ABI of tree attention on the 4-bit cache (include/pasa.h).
#include <algorithm>
#include <cmath>

#include "host_util.cuh"
#include "kv4_tree.cuh"

namespace {

struct TreePlan {
  int row_tiles, ctas;     // ctas: that share all items, or 0: a CTA to a segment
  long long segments;
  size_t part_ml, parts, total;   // workspace: byte offsets and size (part_o is at 0)
};

// With this many items of a segment at most, a CTA takes it whole.
constexpr int kTreeShort = 6;

// Whether the weights of all segments, and grids, fit an int. rows > 0, Sk >= 0.
bool tree_fits(int B, int Hkv, long long rows, int Sk) {
  const long long heads = static_cast<long long>(B) * Hkv, tiles = (rows + pasa::tree::kRows - 1) / pasa::tree::kRows;
  const long long weight = Sk / pasa::tree::kKeys + 2 + pasa::tree::kStart;
  return rows <= INT_MAX - 256 && Sk <= INT_MAX - 256 && heads <= INT_MAX && heads * tiles <= INT_MAX / weight;
}

TreePlan tree_plan(int B, int Hq, int Hkv, int Sq, int Sk, int D) {
  TreePlan pl = {};
  pl.row_tiles = (Hq / Hkv * Sq + pasa::tree::kRows - 1) / pasa::tree::kRows;
  pl.segments = static_cast<long long>(B) * Hkv * pl.row_tiles;
  const int items = 1 + (Sk + pasa::tree::kKeys - 1) / pasa::tree::kKeys;
  if (items <= kTreeShort) return pl;
  pl.ctas = pasa::tree::kCtas;
  const size_t slots = 2 * pasa::tree::kCtas;
  pl.part_ml = slots * D * pasa::tree::kRows * 4;
  pl.parts = pl.part_ml + align_up(slots * pasa::tree::kRows * 8, 256);
  pl.total = pl.parts + align_up(static_cast<size_t>(pl.segments) * 8, 256);
  return pl;
}

template <int D>
int tree_launch(const pasa::tree::Params& p, const TreePlan& pl, cudaStream_t st) {
  static std::atomic<unsigned long long> raised{0};
  const int smem = static_cast<int>(sizeof(pasa::tree::Smem<D>)) + 1024;
  static std::atomic<unsigned long long> asked[2];
  const bool by_segment = pl.segments <= pl.ctas;
  auto merge = by_segment ? pasa::tree::kv4_tree_merge_kernel<D, true> : pasa::tree::kv4_tree_merge_kernel<D, false>;
  if (pl.ctas > 0) prefer_shared(merge, asked[by_segment]);
  const unsigned grid = static_cast<unsigned>(pl.ctas > 0 ? pl.ctas : pl.segments);
  cudaError_t e = launch_clusters(pasa::tree::kv4_tree_kernel<D>, grid, pasa::tree::kThreads, smem, smem, st, false, 1, raised, p);
  if (e == cudaSuccess && pl.ctas > 0) {
    const unsigned places = static_cast<unsigned>(by_segment ? pl.segments : pl.ctas - 1);
    const unsigned fill = p.counts ? static_cast<unsigned>(std::min((p.B + 15) / 16, 64)) : 0;   // for sequences without a node
    e = launch_kernel(merge, dim3(places + fill, D / 8), dim3(256), 0, st, true, p);
  }
  return e == cudaSuccess ? launch_status() : cuda_fail(e);
}

}  // namespace

namespace pasa {
int tree_take_device_error(DeviceError* found) { return take_device_error(found); }
int tree_wait_selftest(cudaStream_t st) { return launch_wait_selftest(st, true); }
}  // namespace pasa

extern "C" {

size_t pasa_attn_fwd_tree_kv4_workspace_bytes(int B, int Hq, int Hkv, int Sq, int Sk, int D) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Sq <= 0 || Sk < 0 || Hq % Hkv != 0 || (D != 64 && D != 128)) return 0;
  if (Sq > pasa::tree::kMaxNodes || !tree_fits(B, Hkv, static_cast<long long>(Hq / Hkv) * Sq, Sk)) return 0;
  return tree_plan(B, Hq, Hkv, Sq, Sk, D).total;
}

int pasa_attn_fwd_tree_kv4(const void* q, const void* k, const void* v, const int* parents, const int* counts, const void* k4,
                           const void* kscale, const void* v4, const void* vscale, const void* shift, const int* lengths, void* o,
                           float* lse, int B, int Hq, int Hkv, int Sq, int Sk, int Sk_cap, int D, float scale, void* workspace,
                           size_t workspace_bytes, void* stream) {
  if (!q || !k || !v || !o) return PASA_ERR_NULLPTR;
  int rc = kv4_validate(k4, kscale, v4, vscale, shift, B, Hkv, Sk_cap, D);
  if (rc != PASA_OK) return rc;
  if (Hq <= 0 || Sq <= 0 || Sk < 0 || Hq % Hkv != 0 || Sk_cap < Sk) return PASA_ERR_SHAPE;
  if (Sq > pasa::tree::kMaxNodes) return PASA_ERR_UNSUPPORTED;
  const long long rows = static_cast<long long>(Hq / Hkv) * Sq;
  if (!tree_fits(B, Hkv, rows, Sk)) return PASA_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse)) return PASA_ERR_ALIGN;
  if (!aligned4(parents) || !aligned4(counts) || !aligned4(lengths)) return PASA_ERR_ALIGN;
  const TreePlan pl = tree_plan(B, Hq, Hkv, Sq, Sk, D);
  if (pl.total > 0) {
    if (!workspace || workspace_bytes < pl.total) return PASA_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return PASA_ERR_ALIGN;
  }
  const unsigned long long q_rows = static_cast<unsigned long long>(B) * Hq * Sq, n_rows = static_cast<unsigned long long>(B) * Hkv * Sq;
  const Kv4Spans c(k4, kscale, v4, vscale, shift, B, Hkv, Sk_cap, D);
  if (any_meet({Span(o, q_rows, 2 * D), Span(lse, q_rows, 4), Span(pl.total ? workspace : nullptr, pl.total, 1)},
               {Span(q, q_rows, 2 * D), Span(k, n_rows, 2 * D), Span(v, n_rows, 2 * D), c.k4, c.kscale, c.v4, c.vscale, c.shift,
                Span(parents, static_cast<unsigned long long>(B) * Sq, 4), Span(counts, B, 4), Span(lengths, B, 4)}))
    return PASA_ERR_SHAPE;
  rc = check_device();
  if (rc != PASA_OK) return rc;
  if (!(scale > 0.0f) || !std::isfinite(scale)) scale = 1.0f / std::sqrt(static_cast<float>(D));
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  pasa::tree::Params p = {};
  p.q = static_cast<const __half*>(q);
  p.k = static_cast<const __half*>(k);
  p.v = static_cast<const __half*>(v);
  p.parents = parents;
  p.counts = counts;
  p.k4 = static_cast<const uint8_t*>(k4);
  p.v4 = static_cast<const uint8_t*>(v4);
  p.kscale = static_cast<const __half*>(kscale);
  p.vscale = static_cast<const __half*>(vscale);
  p.shift = static_cast<const __half*>(shift);
  p.lengths = lengths;
  p.o = static_cast<__half*>(o);
  p.lse = lse;
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + pl.part_ml);
  p.parts = reinterpret_cast<int2*>(ws + pl.parts);
  p.B = B;
  p.Hkv = Hkv;
  p.Sq = Sq;
  p.rows = static_cast<int>(rows);
  p.row_tiles = pl.row_tiles;
  p.Sk = Sk;
  p.cap = Sk_cap;
  p.ctas = pl.ctas;
  p.scale = scale;
  p.scale_log2 = scale * 1.4426950408889634f;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return D == 64 ? tree_launch<64>(p, pl, st) : tree_launch<128>(p, pl, st);
}

}  // extern "C"
