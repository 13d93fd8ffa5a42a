// libpasa.so: the C ABI of rotary positions and of attention over packed prompts (include/pasa.h).
#include <cmath>
#include <cstring>

#include "host_util.cuh"
#include "rope.cuh"

namespace {

// A strided tensor [B, H, S, D] in bytes, for questions of shared memory.
struct Strided {
  uintptr_t at;
  long long stride[3], n[3];   // of the dimensions, largest stride first
  long long row;               // bytes of a row

  Strided(const void* p, const long long* strides, long long B, long long H, long long S, long long D, long long size)
      : at(reinterpret_cast<uintptr_t>(p)), stride{strides[0] * size, strides[1] * size, strides[2] * size}, n{B, H, S}, row(D * size) {
    for (int i = 0; i < 3; ++i)
      if (n[i] == 1) stride[i] = 0;   // a dimension of one has no stride
    for (int i = 0; i < 2; ++i)
      for (int j = 0; j < 2; ++j)
        if (stride[j] < stride[j + 1]) std::swap(stride[j], stride[j + 1]), std::swap(n[j], n[j + 1]);
  }
  // The bytes that dimensions i .. 2 and a row span.
  long long extent(int i) const {
    long long e = row;
    for (; i < 3; ++i) e += (n[i] - 1) * stride[i];
    return e;
  }
  // Whether two of its rows share memory, as far as the strides tell.
  bool folds() const {
    for (int i = 0; i < 3; ++i)
      if (n[i] > 1 && stride[i] < extent(i + 1)) return true;
    return false;
  }
  bool same(const Strided& x) const {
    return at == x.at && row == x.row && std::memcmp(stride, x.stride, sizeof stride) == 0 && std::memcmp(n, x.n, sizeof n) == 0;
  }
  // Whether the two share memory. Two views that lie side by side in one buffer's rows (q and k of a
  // fused projection) do not; other views of one range count as sharing it.
  bool meets(const Strided& x) const {
    const uintptr_t end = at + extent(0), xend = x.at + x.extent(0);
    if (end <= x.at || xend <= at) return false;
    for (int i = 0; i < 3; ++i) {   // the first i strides alike, and what is inside them apart in every period of stride i - 1
      if (stride[i] != x.stride[i] || stride[i] == 0) break;
      const unsigned long long period = static_cast<unsigned long long>(stride[i]);
      if (i > 0 && stride[i - 1] % stride[i] != 0) break;
      const unsigned long long e = extent(i + 1), xe = x.extent(i + 1);
      if (e > period || xe > period) break;
      const unsigned long long d = x.at >= at ? (x.at - at) % period : (period - (at - x.at) % period) % period;
      if (d >= e && d + xe <= period) return false;
    }
    return true;
  }
};

int type_size(int type) { return type == PASA_TYPE_F32 ? 4 : type == PASA_TYPE_F16 || type == PASA_TYPE_BF16 ? 2 : 0; }

// strides: of b, h and s; all at least 0, and their products with the sizes fit 62 bits with room.
bool strides_fit(const long long* strides, long long B, long long H, long long S, long long D) {
  const long long n[3] = {B, H, S};
  long long sum = D;
  for (int i = 0; i < 3; ++i) {
    long long x;
    if (strides[i] < 0) return false;
    if (__builtin_mul_overflow(strides[i], n[i], &x) || __builtin_add_overflow(sum, x, &sum) || sum > (1ll << 58)) return false;
  }
  return true;
}

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

}  // namespace

namespace pasa {
int packed_take_device_error(unsigned long long* info) { return take_device_error(info); }
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
  bool vectors = rotary_dim % 16 == 0 && D % 8 == 0, in_place = true;
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
  p.tokens = static_cast<unsigned>(tokens);
  p.mscale = mscale;
  p.sign = inverse ? -1.0f : 1.0f;
  long long threads;
  if (vectors) {
    p.groups = rotary_dim / 16 + (in_place ? 0 : (D - rotary_dim + 15) / 16);
    // heads of a thread: as many as leave every SM its threads
    p.per = pasa::kRopeHeads;
    while (p.per > 1 && tokens * ((heads + p.per - 1) / p.per) * p.groups < 152ll * 1024) p.per /= 2;
    p.slots = static_cast<unsigned>((heads + p.per - 1) / p.per);
  } else {
    p.groups = rotary_dim / 2 + (in_place ? 0 : D - rotary_dim);
    p.per = 1;
    p.slots = static_cast<unsigned>(heads);
  }
  if (__builtin_mul_overflow(tokens, static_cast<long long>(p.slots) * p.groups, &threads) || threads > 0xFFFFFF00ll - pasa::kRopeThreads)
    return PASA_ERR_SHAPE;
  const int rc = check_device();
  if (rc != PASA_OK) return rc;
  const unsigned grid = static_cast<unsigned>((threads + pasa::kRopeThreads - 1) / pasa::kRopeThreads);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool same = in_type == out_type;
  if (in_type == PASA_TYPE_F16) rope_launch<__half, __half>(p, vectors, interleaved, grid, st);
  else if (in_type == PASA_TYPE_BF16 && same) rope_launch<__nv_bfloat16, __nv_bfloat16>(p, vectors, interleaved, grid, st);
  else if (in_type == PASA_TYPE_BF16) rope_launch<__nv_bfloat16, __half>(p, vectors, interleaved, grid, st);
  else if (same) rope_launch<float, float>(p, vectors, interleaved, grid, st);
  else rope_launch<float, __half>(p, vectors, interleaved, grid, st);
  return launch_status();
}

}  // extern "C"
