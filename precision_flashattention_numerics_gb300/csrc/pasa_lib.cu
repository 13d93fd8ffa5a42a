// libpasa.so: the C ABI declared in include/pasa.h. Host-side argument validation, TMA
// descriptor encoding, workspace layout and kernel dispatch. Compiled as one translation
// unit for sm_103a.
#include <atomic>
#include <climits>
#include <cstddef>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <initializer_list>
#include <utility>
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include "../../include/pasa.h"
#include "attn_fwd.cuh"
#include "attn_fwd2s.cuh"
#include "decode_fwd.cuh"
#include "evict.cuh"
#include "host_util.cuh"
#include "kv4_decode.cuh"
#include "kv4_store.cuh"
#include "kshift.cuh"
#include "ptx.cuh"

namespace pasa {

thread_local int t_last_cuda_error = 0;

// Element i: the FMA-pipe exponential the softmax uses for part of its scores (poly) and the
// MUFU one it uses for the rest (mufu), both of x[i]; pairs go through exp2_fma2 together.
__global__ void exp2_selftest_kernel(const float* __restrict__ x, float* __restrict__ poly, float* __restrict__ mufu,
                                     int n) {
  const int i = 2 * (blockIdx.x * blockDim.x + threadIdx.x);
  if (i >= n) return;
  const float x0 = x[i];
  const float x1 = i + 1 < n ? x[i + 1] : 0.0f;
  float p0, p1;
  exp2_fma2(p0, p1, x0, x1);
  poly[i] = p0;
  mufu[i] = ex2_approx(x0);
  if (i + 1 < n) {
    poly[i + 1] = p1;
    mufu[i + 1] = ex2_approx(x1);
  }
}

}  // namespace pasa

namespace {

bool fp8_mode(int mode) { return mode == PASA_MODE_SHIFT_FP8 || mode == PASA_MODE_NAIVE_FP8; }

// Modes that shift the keys (and so need the block means).
bool shift_mode(int mode) {
  return mode == PASA_MODE_SHIFT_F16ACC || mode == PASA_MODE_SHIFT_F32ACC || mode == PASA_MODE_SHIFT_F16ALL ||
         mode == PASA_MODE_SHIFT_FP8;
}

// Workspace: the keys the attention kernel reads (fp16 K', or e4m3 codes in the FP8 modes),
// the block means [B,Hkv,nb,D] fp16 and, in the FP8 modes, the block scales [B,Hkv,nb] fp32;
// each part 256-byte aligned.
struct WorkspaceLayout {
  size_t kshift_off, means_off, kscale_off, total;
};

WorkspaceLayout workspace_layout(int B, int Hkv, int Sk, int D, int mode) {
  const int bn = pasa::block_rows_for(D);
  const size_t nb = (static_cast<size_t>(Sk) + bn - 1) / bn;
  const size_t eb = fp8_mode(mode) ? 1 : 2;
  WorkspaceLayout w;
  w.kshift_off = 0;
  w.means_off = align_up(static_cast<size_t>(B) * Hkv * Sk * D * eb, 256);
  w.kscale_off = align_up(w.means_off + static_cast<size_t>(B) * Hkv * nb * D * 2, 256);
  w.total = fp8_mode(mode) ? align_up(w.kscale_off + static_cast<size_t>(B) * Hkv * nb * 4, 256) : w.kscale_off;
  return w;
}

template <int D, int OUT, bool PLAIN = false>
int launch_kshift(const void* k, void* ks, void* means, float* kscale, int B, int H, int Sk, cudaStream_t st,
                  int first_block = 0, int cap = 0) {
  constexpr int BN = pasa::block_rows_for(D);
  const int nb = (Sk + BN - 1) / BN;
  if (cap <= 0) cap = Sk;
  dim3 grid(nb - first_block, B * H);
  if constexpr (OUT == pasa::kShiftF16 && !PLAIN) {
    // the fp16 grid-mean shift: the register-resident kernel
    pasa::kshift_reg_kernel<D, BN><<<grid, pasa::kShiftRegThreads, 0, st>>>(
        static_cast<const __half*>(k), static_cast<__half*>(ks), static_cast<__half*>(means), Sk, nb, first_block,
        cap, (cap + BN - 1) / BN);
    cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? PASA_OK : cuda_fail(e);
  }
  pasa::kshift_kernel<D, BN, OUT, PLAIN><<<grid, pasa::kShiftThreads, 0, st>>>(
      static_cast<const __half*>(k), ks, static_cast<__half*>(means), kscale, Sk, nb, first_block, cap,
      (cap + BN - 1) / BN);
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? PASA_OK : cuda_fail(e);
}

// fp16 K' for the fp16 modes; e4m3 codes (of K', or of K in the naive FP8 mode) otherwise.
// The key preparation of `mode` (fp16 shift, or e4m3 codes and scales) for key blocks
// [first_block, ceil(Sk / BN)) of heads holding cap (>= Sk) rows each.
int kshift_dispatch(const void* k, void* ks, void* means, float* kscale, int B, int H, int Sk, int D, int mode,
                    cudaStream_t st, int first_block = 0, int cap = 0) {
  if (mode == PASA_MODE_SHIFT_FP8)
    return launch_kshift<128, pasa::kShiftFp8>(k, ks, means, kscale, B, H, Sk, st, first_block, cap);
  if (mode == PASA_MODE_NAIVE_FP8)
    return launch_kshift<128, pasa::kRawFp8>(k, ks, means, kscale, B, H, Sk, st, first_block, cap);
  return D == 64 ? launch_kshift<64, pasa::kShiftF16>(k, ks, means, nullptr, B, H, Sk, st, first_block, cap)
                 : launch_kshift<128, pasa::kShiftF16>(k, ks, means, nullptr, B, H, Sk, st, first_block, cap);
}

template <int D, bool F16ACC, bool SHIFT, bool CAUSAL, bool STATS, bool F16PV = false, bool FP8 = false>
int launch_attn(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mo,
                const CUtensorMap& mm, const pasa::AttnParams& p, cudaStream_t st, bool pdl = false) {
  constexpr int BN = pasa::block_rows_for(D);
  // ring slots: D = 128 fp16 keys: 3 K + 2 V (201 KB of shared memory); e4m3 keys: 4 + 3
  constexpr int KST = D == 128 ? (FP8 ? 4 : 3) : 4;
  constexpr int VST = D == 128 ? (FP8 ? 3 : 2) : 4;
  using Smem = pasa::AttnSmem<D, BN, KST, VST, FP8>;
  auto kern = pasa::attn_fwd_kernel<D, BN, F16ACC, SHIFT, CAUSAL, KST, VST, STATS, F16PV, FP8>;
  const int smem = static_cast<int>(sizeof(Smem)) + 1024;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return cuda_fail(e);
  const long long ctas = static_cast<long long>(p.n_qblk) * p.Hq * p.B;
  const unsigned splits = p.bps > 0 ? static_cast<unsigned>((p.nbt + p.bps - 1) / p.bps) : 1u;
  e = launch_kernel(kern, dim3(static_cast<unsigned>(ctas), splits), dim3(pasa::kAttnThreads), smem, st, pdl, mq, mk, mv,
                    mo, mm, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? PASA_OK : cuda_fail(e);
}

// The fused-shift kernel (D = 128, modes 0, 1, 4): raw keys in, shift warps in the kernel.
template <bool F16ACC, bool CAUSAL, bool F16PV>
int launch_attn_fused(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mo,
                      const pasa::AttnParams& p, cudaStream_t st) {
  constexpr int D = 128, BN = 128, KST = 3, VST = 2;
  using Smem = pasa::AttnSmem<D, BN, KST, VST, false, true>;
  auto kern = pasa::attn_fwd_kernel<D, BN, F16ACC, true, CAUSAL, KST, VST, false, F16PV, false, true>;
  const int smem = static_cast<int>(sizeof(Smem)) + 1024;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return cuda_fail(e);
  const long long ctas = static_cast<long long>(p.n_qblk) * p.Hq * p.B;
  kern<<<static_cast<unsigned>(ctas), pasa::kAttnThreadsFused, smem, st>>>(mq, mk, mv, mo, mk, p);
  e = cudaGetLastError();
  return e == cudaSuccess ? PASA_OK : cuda_fail(e);
}

template <int D, bool STATS>
int attn_dispatch(int mode, int causal, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                  const CUtensorMap& mo, const CUtensorMap& mm, const pasa::AttnParams& p, cudaStream_t st,
                  bool pdl = false) {
#define PASA_CASE(MODE, F16, SH)                                                        \
  case MODE:                                                                            \
    return causal ? launch_attn<D, F16, SH, true, STATS>(mq, mk, mv, mo, mm, p, st, pdl)     \
                  : launch_attn<D, F16, SH, false, STATS>(mq, mk, mv, mo, mm, p, st, pdl);
  switch (mode) {
    PASA_CASE(PASA_MODE_SHIFT_F16ACC, true, true)
    PASA_CASE(PASA_MODE_SHIFT_F32ACC, false, true)
    PASA_CASE(PASA_MODE_NAIVE_F16ACC, true, false)
    PASA_CASE(PASA_MODE_NOSHIFT_F32ACC, false, false)
    case PASA_MODE_SHIFT_F16ALL:
      return causal ? launch_attn<D, true, true, true, STATS, true>(mq, mk, mv, mo, mm, p, st, pdl)
                    : launch_attn<D, true, true, false, STATS, true>(mq, mk, mv, mo, mm, p, st, pdl);
    case PASA_MODE_SHIFT_FP8:
    case PASA_MODE_NAIVE_FP8:
      if constexpr (D == 128 && !STATS) {
        if (mode == PASA_MODE_SHIFT_FP8)
          return causal ? launch_attn<D, false, true, true, false, false, true>(mq, mk, mv, mo, mm, p, st, pdl)
                        : launch_attn<D, false, true, false, false, false, true>(mq, mk, mv, mo, mm, p, st, pdl);
        return causal ? launch_attn<D, false, false, true, false, false, true>(mq, mk, mv, mo, mm, p, st, pdl)
                      : launch_attn<D, false, false, false, false, false, true>(mq, mk, mv, mo, mm, p, st, pdl);
      }
      return PASA_ERR_UNSUPPORTED;
    default:
      return PASA_ERR_UNSUPPORTED;
  }
#undef PASA_CASE
}

int validate_shape(int B, int Hq, int Hkv, int Sq, int Sk, int D, int mode) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Sq <= 0 || Sk <= 0 || Hq % Hkv != 0) return PASA_ERR_SHAPE;
  if (D != 64 && D != 128) return PASA_ERR_UNSUPPORTED;
  if (mode < PASA_MODE_SHIFT_F16ACC || mode > PASA_MODE_NAIVE_FP8) return PASA_ERR_UNSUPPORTED;
  if (fp8_mode(mode) && D != 128) return PASA_ERR_UNSUPPORTED;
  // grid size, TMA plane counts and flat LSE indices fit in 32-bit signed integers
  const long long n_qblk = (static_cast<long long>(Sq) + pasa::kTileRows - 1) / pasa::kTileRows;
  if (n_qblk * Hq * B > 0x7fffffffLL) return PASA_ERR_SHAPE;
  if (static_cast<long long>(B) * Hq > 0x7fffffffLL || static_cast<long long>(B) * Hkv > 0x7fffffffLL)
    return PASA_ERR_SHAPE;
  return PASA_OK;
}

int validate(const void* q, const void* k, const void* v, const void* o, const float* lse, int B, int Hq, int Hkv,
             int Sq, int Sk, int D, int mode) {
  if (!q || !k || !v || !o) return PASA_ERR_NULLPTR;
  const int rc = validate_shape(B, Hq, Hkv, Sq, Sk, D, mode);
  if (rc != PASA_OK) return rc;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || (lse && !aligned16(lse)))
    return PASA_ERR_ALIGN;
  return PASA_OK;
}

// D = 64 prefill, modes 0-3: two softmax warp sets on alternate key blocks.
template <bool F16ACC, bool SHIFT, bool CAUSAL>
int launch_2set(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mo,
                const CUtensorMap& mm, const pasa::AttnParams& p, cudaStream_t st, bool pdl = false) {
  constexpr int KST = 4, VST = 4;
  auto kern = pasa::twoset::attn_fwd_2set_kernel<64, 128, F16ACC, SHIFT, CAUSAL, KST, VST, false>;
  const int smem = static_cast<int>(sizeof(pasa::twoset::AttnSmem<64, 128, KST, VST>)) + 1024;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return cuda_fail(e);
  const long long ctas = static_cast<long long>(p.n_qblk) * p.Hq * p.B;
  e = launch_kernel(kern, dim3(static_cast<unsigned>(ctas)), dim3(pasa::twoset::kAttnThreads), smem, st, pdl, mq, mk,
                    mv, mo, mm, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? PASA_OK : cuda_fail(e);
}

int twoset_dispatch(int mode, int causal, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                    const CUtensorMap& mo, const CUtensorMap& mm, const pasa::AttnParams& p, cudaStream_t st,
                    bool pdl = false) {
#define PASA_2S_CASE(MODE, F16, SH)                                                   \
  case MODE:                                                                          \
    return causal ? launch_2set<F16, SH, true>(mq, mk, mv, mo, mm, p, st, pdl)        \
                  : launch_2set<F16, SH, false>(mq, mk, mv, mo, mm, p, st, pdl);
  switch (mode) {
    PASA_2S_CASE(PASA_MODE_SHIFT_F16ACC, true, true)
    PASA_2S_CASE(PASA_MODE_SHIFT_F32ACC, false, true)
    PASA_2S_CASE(PASA_MODE_NAIVE_F16ACC, true, false)
    PASA_2S_CASE(PASA_MODE_NOSHIFT_F32ACC, false, false)
    default:
      return PASA_ERR_UNSUPPORTED;
  }
#undef PASA_2S_CASE
}

// The swapped-operand decode kernel (D = 128, at most 32 packed query rows per kv head).
// pdl: launch with programmatic stream serialization, so the kernel may start while the
// refresh queued ahead of it still runs (it waits for it before reading p.dep_block on).
template <int NQ, bool F16ACC, bool SHIFT, bool F16PV, bool FP8 = false>
int launch_decode(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mm,
                         const pasa::DecodeParams& p, long long planes, int splits, cudaStream_t st, bool pdl) {
  // e4m3 keys at 16 columns: two softmax warpgroups (even and odd key blocks) and rings of
  // 4 K + 3 V; fp16 keys: one group with 3 K' + 3 V (16 columns) or 3 + 2 (32 columns).
  // (Measured on the 8 x 32K-key cache: two groups lift the e4m3 cache by 7%, while the fp16
  // cache gains more from the third V slot that two groups leave no room for.)
  constexpr int G = (FP8 && NQ == 16) ? 2 : 1;
  constexpr int KST = FP8 ? 4 : 3, VST = (FP8 || NQ == 16) ? 3 : 2;
  auto kern = pasa::decode_fwd_kernel<NQ, F16ACC, SHIFT, F16PV, KST, VST, FP8, G>;
  const int smem = static_cast<int>(sizeof(pasa::DecodeSmem<NQ, KST, VST, FP8, G>)) + 1024;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return cuda_fail(e);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(planes), static_cast<unsigned>(splits));
  cfg.blockDim = dim3(pasa::dec_threads(G));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  unsigned na = 0;
  if (p.cluster) {
    // the splits of a kv head as one cluster (at most 8: the portable cluster size)
    attr[na].id = cudaLaunchAttributeClusterDimension;
    attr[na].val.clusterDim.x = 1;
    attr[na].val.clusterDim.y = static_cast<unsigned>(splits);
    attr[na].val.clusterDim.z = 1;
    ++na;
  }
  if (pdl) {
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
  }
  if (na > 0) {
    cfg.attrs = attr;
    cfg.numAttrs = na;
  }
  e = cudaLaunchKernelEx(&cfg, kern, mq, mk, mv, mm, p);
  if (e != cudaSuccess) return cuda_fail(e);
  e = cudaGetLastError();
  return e == cudaSuccess ? PASA_OK : cuda_fail(e);
}

template <int NQ>
int decode_dispatch(int mode, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                           const CUtensorMap& mm, const pasa::DecodeParams& p, long long planes, int splits,
                           cudaStream_t st, bool pdl) {
#define PASA_DEC_CASE(MODE, ...) \
  case MODE: return launch_decode<NQ, __VA_ARGS__>(mq, mk, mv, mm, p, planes, splits, st, pdl);
  switch (mode) {
    PASA_DEC_CASE(PASA_MODE_SHIFT_F16ACC, true, true, false)
    PASA_DEC_CASE(PASA_MODE_SHIFT_F32ACC, false, true, false)
    PASA_DEC_CASE(PASA_MODE_NAIVE_F16ACC, true, false, false)
    PASA_DEC_CASE(PASA_MODE_NOSHIFT_F32ACC, false, false, false)
    PASA_DEC_CASE(PASA_MODE_SHIFT_F16ALL, true, true, true)
    PASA_DEC_CASE(PASA_MODE_SHIFT_FP8, false, true, false, true)
    PASA_DEC_CASE(PASA_MODE_NAIVE_FP8, false, false, false, true)
    default: return PASA_ERR_UNSUPPORTED;
  }
#undef PASA_DEC_CASE
}

}  // namespace

extern "C" {

int pasa_block_rows(int D) { return pasa::block_rows_for(D); }

int pasa_last_cuda_error(void) { return t_last_cuda_error; }

int pasa_device_supported(int device) {
  int major = 0, minor = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, device) != cudaSuccess) return 0;
  return (major == 10 && minor == 3) ? 1 : 0;
}

const char* pasa_strerror(int status) {
  switch (status) {
    case PASA_OK: return "ok";
    case PASA_ERR_NULLPTR: return "a required pointer is NULL";
    case PASA_ERR_SHAPE: return "invalid sizes (<= 0, Hq % Hkv != 0, or too large)";
    case PASA_ERR_UNSUPPORTED: return "unsupported head dim, mode or device (needs D in {64,128}, sm_103)";
    case PASA_ERR_ALIGN: return "a pointer is not 16-byte aligned";
    case PASA_ERR_CUDA: return "a CUDA call failed";
    case PASA_ERR_TIMEOUT: return "a device pipeline wait timed out";
    case PASA_ERR_WORKSPACE: return "workspace missing or too small";
    default: return "unknown status";
  }
}

size_t pasa_attn_fwd_workspace_bytes(int B, int Hkv, int Sk, int D, int mode) {
  if (B <= 0 || Hkv <= 0 || Sk <= 0 || pasa::block_rows_for(D) == 0) return 0;
  if (!shift_mode(mode) && !fp8_mode(mode)) return 0;
  if (fp8_mode(mode) && D != 128) return 0;
  return workspace_layout(B, Hkv, Sk, D, mode).total;
}

int pasa_kshift(const void* k, void* k_shifted, void* means, int B, int H, int Sk, int D, void* stream) {
  if (!k || !k_shifted || !means) return PASA_ERR_NULLPTR;
  if (B <= 0 || H <= 0 || Sk <= 0) return PASA_ERR_SHAPE;
  if (D != 64 && D != 128) return PASA_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * H > 65535) return PASA_ERR_SHAPE;  // grid.y
  if (!aligned16(k) || !aligned16(k_shifted) || !aligned16(means)) return PASA_ERR_ALIGN;
  int rc = check_device();
  if (rc != PASA_OK) return rc;
  return kshift_dispatch(k, k_shifted, means, nullptr, B, H, Sk, D, PASA_MODE_SHIFT_F16ACC,
                         static_cast<cudaStream_t>(stream));
}

int pasa_kshift_mean(const void* k, void* k_shifted, void* means, int B, int H, int Sk, int D, int mean_rule,
                     void* stream) {
  if (mean_rule == PASA_MEAN_GRID) return pasa_kshift(k, k_shifted, means, B, H, Sk, D, stream);
  if (mean_rule != PASA_MEAN_PLAIN) return PASA_ERR_UNSUPPORTED;
  if (!k || !k_shifted || !means) return PASA_ERR_NULLPTR;
  if (B <= 0 || H <= 0 || Sk <= 0) return PASA_ERR_SHAPE;
  if (D != 64 && D != 128) return PASA_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * H > 65535) return PASA_ERR_SHAPE;  // grid.y
  if (!aligned16(k) || !aligned16(k_shifted) || !aligned16(means)) return PASA_ERR_ALIGN;
  int rc = check_device();
  if (rc != PASA_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return D == 64 ? launch_kshift<64, pasa::kShiftF16, true>(k, k_shifted, means, nullptr, B, H, Sk, st)
                 : launch_kshift<128, pasa::kShiftF16, true>(k, k_shifted, means, nullptr, B, H, Sk, st);
}

int pasa_kprep_fp8(const void* k, void* k8, void* means, float* kscale, int B, int H, int Sk, int D, int mode,
                   void* stream) {
  if (!k || !k8 || !kscale || (mode == PASA_MODE_SHIFT_FP8 && !means)) return PASA_ERR_NULLPTR;
  if (B <= 0 || H <= 0 || Sk <= 0) return PASA_ERR_SHAPE;
  if (D != 128 || !fp8_mode(mode)) return PASA_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * H > 65535) return PASA_ERR_SHAPE;  // grid.y
  if (!aligned16(k) || !aligned16(k8) || (means && !aligned16(means)) || !aligned16(kscale)) return PASA_ERR_ALIGN;
  int rc = check_device();
  if (rc != PASA_OK) return rc;
  return kshift_dispatch(k, k8, means, kscale, B, H, Sk, D, mode, static_cast<cudaStream_t>(stream));
}

int pasa_kshift_blocks(const void* k, void* k_shifted, void* means, int B, int H, int Sk, int Sk_cap, int D,
                       int first_block, void* stream) {
  if (!k || !k_shifted || !means) return PASA_ERR_NULLPTR;
  if (B <= 0 || H <= 0 || Sk <= 0 || Sk_cap < Sk) return PASA_ERR_SHAPE;
  if (D != 64 && D != 128) return PASA_ERR_UNSUPPORTED;
  const int nb = (Sk + pasa::block_rows_for(D) - 1) / pasa::block_rows_for(D);
  if (first_block < 0 || first_block >= nb) return PASA_ERR_SHAPE;
  if (static_cast<long long>(B) * H > 65535) return PASA_ERR_SHAPE;  // grid.y
  if (!aligned16(k) || !aligned16(k_shifted) || !aligned16(means)) return PASA_ERR_ALIGN;
  int rc = check_device();
  if (rc != PASA_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return D == 64 ? launch_kshift<64, pasa::kShiftF16>(k, k_shifted, means, nullptr, B, H, Sk, st, first_block, Sk_cap)
                 : launch_kshift<128, pasa::kShiftF16>(k, k_shifted, means, nullptr, B, H, Sk, st, first_block, Sk_cap);
}

// Launch the attention kernel on (possibly shifted) keys `kk` and block means `mm`.
// pdl: the key preparation of the same call was launched just before on `st` (see
// launch_kernel); never with the diagnostic outputs, whose zeroing sits in between.
static int attn_launch(const void* q, const void* kk, const void* mm, const void* v, void* o, float* lse, int B,
                       int Hq, int Hkv, int Sq, int Sk, int D, int causal, float scale, int mode, cudaStream_t st,
                       float* stats = nullptr, float* block_stats = nullptr, const float* kscale = nullptr,
                       bool pdl = false) {
  const bool shift = shift_mode(mode);
  if (!(scale > 0.0f) || !std::isfinite(scale)) scale = 1.0f / std::sqrt(static_cast<float>(D));
  const int bn = pasa::block_rows_for(D);
  const int nb = (Sk + bn - 1) / bn;
  int rc;
  CUtensorMap mq, mk, mv, mo, mmeans;
  if ((rc = make_map(&mq, q, D, Sq, static_cast<long long>(B) * Hq, pasa::kTileRows)) != PASA_OK) return rc;
  if ((rc = make_map(&mk, kk, D, Sk, static_cast<long long>(B) * Hkv, bn, fp8_mode(mode) ? 1 : 2)) != PASA_OK)
    return rc;
  if ((rc = make_map(&mv, v, D, Sk, static_cast<long long>(B) * Hkv, bn)) != PASA_OK) return rc;
  if ((rc = make_map(&mo, o, D, Sq, static_cast<long long>(B) * Hq, pasa::kTileRows)) != PASA_OK) return rc;
  if (shift) {
    if ((rc = make_map(&mmeans, mm, D, nb, static_cast<long long>(B) * Hkv, pasa::kChunkBlocks)) != PASA_OK)
      return rc;
  } else {
    mmeans = mk;  // unused by the no-shift kernels
  }
  pasa::AttnParams p;
  p.lse = lse;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.Sq = Sq;
  p.Sk = Sk;
  p.n_qblk = (Sq + pasa::kTileRows - 1) / pasa::kTileRows;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.inv_scale_log2 = 1.0f / p.scale_log2;
  p.stats = stats;
  p.bstats = reinterpret_cast<unsigned*>(block_stats);
  p.nbt = nb;
  p.kscale = kscale;
  p.sq_mod = Sq;
  p.bps = 0;
  p.part_o = nullptr;
  p.part_lse = nullptr;
  p.kshift_out = nullptr;
  p.means_out = nullptr;
  if (block_stats) {
    const cudaError_t e = cudaMemsetAsync(block_stats, 0, static_cast<size_t>(B) * Hq * nb * 2 * sizeof(float), st);
    if (e != cudaSuccess) return cuda_fail(e);
  }
  if (stats)
    return D == 64 ? attn_dispatch<64, true>(mode, causal, mq, mk, mv, mo, mmeans, p, st)
                   : attn_dispatch<128, true>(mode, causal, mq, mk, mv, mo, mmeans, p, st);
  if (D == 64 && mode <= PASA_MODE_NOSHIFT_F32ACC)
    return twoset_dispatch(mode, causal, mq, mk, mv, mo, mmeans, p, st, pdl);
  return D == 64 ? attn_dispatch<64, false>(mode, causal, mq, mk, mv, mo, mmeans, p, st, pdl)
                 : attn_dispatch<128, false>(mode, causal, mq, mk, mv, mo, mmeans, p, st, pdl);
}

int pasa_attn_fwd_shifted(const void* q, const void* k_shifted, const void* means, const void* v, void* o,
                          float* lse, int B, int Hq, int Hkv, int Sq, int Sk, int D, int causal, float scale,
                          int mode, void* stream) {
  int rc = validate(q, k_shifted, v, o, lse, B, Hq, Hkv, Sq, Sk, D, mode);
  if (rc != PASA_OK) return rc;
  if (fp8_mode(mode)) return PASA_ERR_UNSUPPORTED;  // the FP8 modes read e4m3 keys, not fp16 K'
  const bool shift = shift_mode(mode);
  if (shift && !means) return PASA_ERR_NULLPTR;
  if (shift && !aligned16(means)) return PASA_ERR_ALIGN;
  rc = check_device();
  if (rc != PASA_OK) return rc;
  return attn_launch(q, k_shifted, shift ? means : k_shifted, v, o, lse, B, Hq, Hkv, Sq, Sk, D, causal, scale, mode,
                     static_cast<cudaStream_t>(stream));
}

int pasa_attn_fwd_fp8(const void* q, const void* k8, const void* means, const float* kscale, const void* v, void* o,
                      float* lse, int B, int Hq, int Hkv, int Sq, int Sk, int D, int causal, float scale, int mode,
                      void* stream) {
  int rc = validate(q, k8, v, o, lse, B, Hq, Hkv, Sq, Sk, D, mode);
  if (rc != PASA_OK) return rc;
  if (!fp8_mode(mode)) return PASA_ERR_UNSUPPORTED;
  if (!kscale || (mode == PASA_MODE_SHIFT_FP8 && !means)) return PASA_ERR_NULLPTR;
  if (!aligned16(kscale) || (means && !aligned16(means))) return PASA_ERR_ALIGN;
  rc = check_device();
  if (rc != PASA_OK) return rc;
  return attn_launch(q, k8, mode == PASA_MODE_SHIFT_FP8 ? means : k8, v, o, lse, B, Hq, Hkv, Sq, Sk, D, causal, scale,
                     mode, static_cast<cudaStream_t>(stream), nullptr, nullptr, kscale);
}

// Decode path: key-block split and its partial-result workspace. By default at most one
// wave of CTAs (152 SMs, one CTA each) and at least eight key blocks per split, so that a
// CTA's fixed start-up and pipeline fill stay small against its streaming time.
static int decode_split(int B, int Hkv, int Sk, int D, int splits_req, int* splits_out) {
  const int bn = pasa::block_rows_for(D);
  const int nb = (Sk + bn - 1) / bn;
  const long long units = static_cast<long long>(B) * Hkv;
  int splits = splits_req > 0 ? splits_req : static_cast<int>(std::min<long long>(152 / units, nb / 8));
  splits = std::max(1, std::min(std::min(splits, nb), 65535));   // grid.y
  const int bps = (nb + splits - 1) / splits;
  splits = (nb + bps - 1) / bps;
  *splits_out = splits;
  return splits > 1 ? bps : 0;
}

// The swapped-operand decode kernel merges up to 8 splits of a kv head inside one cluster.
static bool decode_cluster_merge(int D, long long rows, int splits) {
  return D == 128 && rows <= 32 && splits >= 2 && splits <= 8;
}

size_t pasa_attn_fwd_decode_workspace_bytes(int B, int Hq, int Hkv, int Sq, int Sk, int D, int splits) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Sq <= 0 || Sk <= 0 || Hq % Hkv != 0 || pasa::block_rows_for(D) == 0) return 0;
  int sp = 1;
  if (decode_split(B, Hkv, Sk, D, splits, &sp) == 0) return 0;
  if (decode_cluster_merge(D, static_cast<long long>(Hq / Hkv) * Sq, sp)) return 0;
  const size_t rows = static_cast<size_t>(B) * Hq * Sq;
  return align_up(static_cast<size_t>(sp) * rows * D * 4, 256) + align_up(static_cast<size_t>(sp) * rows * 4, 256);
}

// Decode on a key cache: fp16 keys (K' or K) for modes 0-4, e4m3 codes with block scales
// `kscale` for modes 5 and 6. dep_block < nb: the kernel queued just ahead on the stream
// rewrites key blocks [dep_block, nb) (a refresh); the swapped-operand decode kernel then
// starts while it runs and waits for it only before reading those blocks.
static int decode_impl(const void* q, const void* k_shifted, const void* means, const float* kscale, const void* v,
                       void* o, float* lse, int B, int Hq, int Hkv, int Sq, int Sk, int Sk_cap, int D, int causal,
                       float scale, int mode, int splits, void* workspace, size_t workspace_bytes, void* stream,
                       int dep_block = INT_MAX) {
  int rc = validate(q, k_shifted, v, o, lse, B, Hq, Hkv, Sq, Sk, D, mode);
  if (rc != PASA_OK) return rc;
  if (Sk_cap < Sk) return PASA_ERR_SHAPE;
  if (splits < 0) return PASA_ERR_UNSUPPORTED;
  const int g = Hq / Hkv;
  if (static_cast<long long>(g) * Sq > pasa::kTileRows) return PASA_ERR_UNSUPPORTED;  // one tile per kv group
  const bool fp8 = fp8_mode(mode);
  // e4m3 keys run on the swapped-operand decode kernel only (D = 128, up to 32 packed rows)
  if (fp8 && (D != 128 || static_cast<long long>(g) * Sq > 32)) return PASA_ERR_UNSUPPORTED;
  if (fp8 && !kscale) return PASA_ERR_NULLPTR;
  if (fp8 && !aligned16(kscale)) return PASA_ERR_ALIGN;
  const bool shift = shift_mode(mode);
  if (shift && !means) return PASA_ERR_NULLPTR;
  if (shift && !aligned16(means)) return PASA_ERR_ALIGN;
  int sp = 1;
  const int bps = decode_split(B, Hkv, Sk, D, splits, &sp);
  const size_t need = pasa_attn_fwd_decode_workspace_bytes(B, Hq, Hkv, Sq, Sk, D, splits);
  const bool cluster = bps > 0 && decode_cluster_merge(D, static_cast<long long>(g) * Sq, sp);
  if (bps > 0 && !cluster) {
    if (!workspace || workspace_bytes < need) return PASA_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return PASA_ERR_ALIGN;
  }
  rc = check_device();
  if (rc != PASA_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!(scale > 0.0f) || !std::isfinite(scale)) scale = 1.0f / std::sqrt(static_cast<float>(D));
  const int bn = pasa::block_rows_for(D);
  const int nb = (Sk + bn - 1) / bn;
  // Q and O viewed as [B * Hkv, g * Sq, D]: the query rows of a kv group's g heads, contiguous
  const int rows = g * Sq;
  const long long planes = static_cast<long long>(B) * Hkv;
  const size_t nrows = static_cast<size_t>(B) * Hq * Sq;
  float* part_o = nullptr;
  float* part_lse = nullptr;
  if (bps > 0 && !cluster) {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    part_o = reinterpret_cast<float*>(ws);
    part_lse = reinterpret_cast<float*>(ws + align_up(static_cast<size_t>(sp) * nrows * D * 4, 256));
  }
  CUtensorMap mq, mk, mv, mo, mmeans;
  // the cache: Sk valid rows of Sk_cap per head (reads past Sk are zero-filled and masked)
  if ((rc = make_map(&mk, k_shifted, D, Sk, planes, bn, fp8 ? 1 : 2, Sk_cap)) != PASA_OK) return rc;
  if ((rc = make_map(&mv, v, D, Sk, planes, bn, 2, Sk_cap)) != PASA_OK) return rc;
  if (shift) {
    if ((rc = make_map(&mmeans, means, D, nb, planes, pasa::kChunkBlocks, 2, (Sk_cap + bn - 1) / bn)) != PASA_OK)
      return rc;
  } else {
    mmeans = mk;
  }
  if (D == 128 && rows <= 32) {
    // few rows: keys on the MMA's M side (decode_fwd_kernel)
    const int nq = rows <= 16 ? 16 : 32;
    if ((rc = make_map(&mq, q, D, rows, planes, nq)) != PASA_OK) return rc;
    pasa::DecodeParams dp;
    dp.o = static_cast<__half*>(o);
    dp.lse = lse;
    dp.part_o = part_o;
    dp.part_lse = part_lse;
    dp.rows = rows;
    dp.sq = Sq;
    dp.Sk = Sk;
    dp.nbt = nb;
    dp.bps = bps;
    dp.causal = causal ? 1 : 0;
    dp.scale_log2 = scale * 1.4426950408889634f;
    dp.cluster = cluster ? 1 : 0;
    dp.kscale = kscale;
    dp.kstride = (Sk_cap + bn - 1) / bn;
    dp.dep_block = dep_block;
    const bool pdl = dep_block < nb;
    rc = nq == 16 ? decode_dispatch<16>(mode, mq, mk, mv, mmeans, dp, planes, sp, st, pdl)
                  : decode_dispatch<32>(mode, mq, mk, mv, mmeans, dp, planes, sp, st, pdl);
  } else {
    // query rows on the MMA's M side: the attention kernel on the packed [g * Sq] rows
    if ((rc = make_map(&mq, q, D, rows, planes, pasa::kTileRows)) != PASA_OK) return rc;
    if ((rc = make_map(&mo, o, D, rows, planes, pasa::kTileRows)) != PASA_OK) return rc;
    pasa::AttnParams p;
    p.lse = lse;
    p.B = B;
    p.Hq = Hkv;
    p.Hkv = Hkv;
    p.Sq = rows;
    p.Sk = Sk;
    p.n_qblk = 1;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.inv_scale_log2 = 1.0f / p.scale_log2;
    p.stats = nullptr;
    p.bstats = nullptr;
    p.nbt = nb;
    p.kscale = nullptr;
    p.sq_mod = Sq;
    p.bps = bps;
    p.part_o = part_o;
    p.part_lse = part_lse;
    p.kshift_out = nullptr;
    p.means_out = nullptr;
    rc = D == 64 ? attn_dispatch<64, false>(mode, causal, mq, mk, mv, mo, mmeans, p, st)
                 : attn_dispatch<128, false>(mode, causal, mq, mk, mv, mo, mmeans, p, st);
  }
  if (rc != PASA_OK || bps == 0 || cluster) return rc;
  const unsigned cblocks = static_cast<unsigned>((nrows + 7) / 8);
  if (D == 64)
    pasa::combine_splits_kernel<64><<<cblocks, 256, 0, st>>>(part_o, part_lse, sp, static_cast<long long>(nrows),
                                                             static_cast<__half*>(o), lse);
  else
    pasa::combine_splits_kernel<128><<<cblocks, 256, 0, st>>>(part_o, part_lse, sp, static_cast<long long>(nrows),
                                                              static_cast<__half*>(o), lse);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? PASA_OK : cuda_fail(e);
}

int pasa_attn_fwd_decode(const void* q, const void* k_shifted, const void* means, const void* v, void* o, float* lse,
                         int B, int Hq, int Hkv, int Sq, int Sk, int Sk_cap, int D, int causal, float scale, int mode,
                         int splits, void* workspace, size_t workspace_bytes, void* stream) {
  if (fp8_mode(mode)) return PASA_ERR_UNSUPPORTED;   // e4m3 caches: pasa_attn_fwd_decode_fp8
  return decode_impl(q, k_shifted, means, nullptr, v, o, lse, B, Hq, Hkv, Sq, Sk, Sk_cap, D, causal, scale, mode,
                     splits, workspace, workspace_bytes, stream);
}

int pasa_attn_fwd_decode_step(const void* q, const void* k, void* k_shifted, void* means, const void* v, void* o,
                              float* lse, int B, int Hq, int Hkv, int Sq, int Sk, int Sk_cap, int D, int causal,
                              float scale, int mode, int first_block, int splits, void* workspace,
                              size_t workspace_bytes, void* stream) {
  if (fp8_mode(mode)) return PASA_ERR_UNSUPPORTED;   // e4m3 caches: pasa_kprep_fp8_blocks + _decode_fp8
  if (!shift_mode(mode)) {
    // raw-key modes keep no shifted copy: nothing to refresh
    return decode_impl(q, k_shifted, means, nullptr, v, o, lse, B, Hq, Hkv, Sq, Sk, Sk_cap, D, causal, scale, mode,
                       splits, workspace, workspace_bytes, stream);
  }
  // argument checks of both calls before anything is enqueued
  if (!k) return PASA_ERR_NULLPTR;
  if (!aligned16(k)) return PASA_ERR_ALIGN;
  int rc = validate(q, k_shifted, v, o, lse, B, Hq, Hkv, Sq, Sk, D, mode);
  if (rc != PASA_OK) return rc;
  if (!means) return PASA_ERR_NULLPTR;
  if (!aligned16(means)) return PASA_ERR_ALIGN;
  if (Sk_cap < Sk || splits < 0) return Sk_cap < Sk ? PASA_ERR_SHAPE : PASA_ERR_UNSUPPORTED;
  const int nb = (Sk + pasa::block_rows_for(D) - 1) / pasa::block_rows_for(D);
  if (first_block < 0 || first_block >= nb || static_cast<long long>(B) * Hkv > 65535) return PASA_ERR_SHAPE;
  if (static_cast<long long>(Hq / Hkv) * Sq > pasa::kTileRows) return PASA_ERR_UNSUPPORTED;
  int sp = 1;
  const int bps = decode_split(B, Hkv, Sk, D, splits, &sp);
  if (bps > 0 && !decode_cluster_merge(D, static_cast<long long>(Hq / Hkv) * Sq, sp)) {
    if (!workspace || workspace_bytes < pasa_attn_fwd_decode_workspace_bytes(B, Hq, Hkv, Sq, Sk, D, splits))
      return PASA_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return PASA_ERR_ALIGN;
  }
  rc = pasa_kshift_blocks(k, k_shifted, means, B, Hkv, Sk, Sk_cap, D, first_block, stream);
  if (rc != PASA_OK) return rc;
  return decode_impl(q, k_shifted, means, nullptr, v, o, lse, B, Hq, Hkv, Sq, Sk, Sk_cap, D, causal, scale, mode,
                     splits, workspace, workspace_bytes, stream, first_block);
}

int pasa_attn_fwd_decode_step_fp8(const void* q, const void* k, void* k8, void* means, float* kscale, const void* v,
                                  void* o, float* lse, int B, int Hq, int Hkv, int Sq, int Sk, int Sk_cap, int D,
                                  int causal, float scale, int mode, int first_block, int splits, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  if (!fp8_mode(mode)) return PASA_ERR_UNSUPPORTED;   // fp16 caches: pasa_attn_fwd_decode_step
  // argument checks of both calls before anything is enqueued
  if (!k || !kscale || (mode == PASA_MODE_SHIFT_FP8 && !means)) return PASA_ERR_NULLPTR;
  if (!aligned16(k) || !aligned16(kscale) || (means && !aligned16(means))) return PASA_ERR_ALIGN;
  int rc = validate(q, k8, v, o, lse, B, Hq, Hkv, Sq, Sk, D, mode);
  if (rc != PASA_OK) return rc;
  if (D != 128 || static_cast<long long>(Hq / Hkv) * Sq > 32) return PASA_ERR_UNSUPPORTED;
  if (Sk_cap < Sk || splits < 0) return Sk_cap < Sk ? PASA_ERR_SHAPE : PASA_ERR_UNSUPPORTED;
  const int nb = (Sk + 127) / 128;
  if (first_block < 0 || first_block >= nb || static_cast<long long>(B) * Hkv > 65535) return PASA_ERR_SHAPE;
  int sp = 1;
  const int bps = decode_split(B, Hkv, Sk, D, splits, &sp);
  if (bps > 0 && !decode_cluster_merge(D, static_cast<long long>(Hq / Hkv) * Sq, sp)) {
    if (!workspace || workspace_bytes < pasa_attn_fwd_decode_workspace_bytes(B, Hq, Hkv, Sq, Sk, D, splits))
      return PASA_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return PASA_ERR_ALIGN;
  }
  rc = pasa_kprep_fp8_blocks(k, k8, means, kscale, B, Hkv, Sk, Sk_cap, D, mode, first_block, stream);
  if (rc != PASA_OK) return rc;
  return decode_impl(q, k8, means, kscale, v, o, lse, B, Hq, Hkv, Sq, Sk, Sk_cap, D, causal, scale, mode, splits,
                     workspace, workspace_bytes, stream, first_block);
}

int pasa_attn_fwd_decode_fp8(const void* q, const void* k8, const void* means, const float* kscale, const void* v,
                             void* o, float* lse, int B, int Hq, int Hkv, int Sq, int Sk, int Sk_cap, int D, int causal,
                             float scale, int mode, int splits, void* workspace, size_t workspace_bytes, void* stream) {
  if (!fp8_mode(mode)) return PASA_ERR_UNSUPPORTED;
  return decode_impl(q, k8, means, kscale, v, o, lse, B, Hq, Hkv, Sq, Sk, Sk_cap, D, causal, scale, mode, splits,
                     workspace, workspace_bytes, stream);
}

int pasa_kprep_fp8_blocks(const void* k, void* k8, void* means, float* kscale, int B, int H, int Sk, int Sk_cap, int D,
                          int mode, int first_block, void* stream) {
  if (!k || !k8 || !kscale || (mode == PASA_MODE_SHIFT_FP8 && !means)) return PASA_ERR_NULLPTR;
  if (B <= 0 || H <= 0 || Sk <= 0 || Sk_cap < Sk) return PASA_ERR_SHAPE;
  if (D != 128 || !fp8_mode(mode)) return PASA_ERR_UNSUPPORTED;
  const int nb = (Sk + 127) / 128;
  if (first_block < 0 || first_block >= nb) return PASA_ERR_SHAPE;
  if (static_cast<long long>(B) * H > 65535) return PASA_ERR_SHAPE;  // grid.y
  if (!aligned16(k) || !aligned16(k8) || !aligned16(kscale) || (means && !aligned16(means))) return PASA_ERR_ALIGN;
  int rc = check_device();
  if (rc != PASA_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return mode == PASA_MODE_SHIFT_FP8
             ? launch_kshift<128, pasa::kShiftFp8>(k, k8, means, kscale, B, H, Sk, st, first_block, Sk_cap)
             : launch_kshift<128, pasa::kRawFp8>(k, k8, means, kscale, B, H, Sk, st, first_block, Sk_cap);
}

int pasa_attn_fwd_ws(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv,
                     int Sq, int Sk, int D, int causal, float scale, int mode, void* workspace,
                     size_t workspace_bytes, void* stream) {
  int rc = validate(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, D, mode);
  if (rc != PASA_OK) return rc;
  const bool prep = shift_mode(mode) || fp8_mode(mode);  // the shift kernel runs first
  const WorkspaceLayout wl = workspace_layout(B, Hkv, Sk, D, mode);
  if (prep) {
    if (!workspace || workspace_bytes < wl.total) return PASA_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return PASA_ERR_ALIGN;
    if (static_cast<long long>(B) * Hkv > 65535) return PASA_ERR_SHAPE;  // kshift grid.y
  }
  rc = check_device();
  if (rc != PASA_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const void* kk = k;
  const void* mm = k;
  float* kscale = nullptr;
  if (prep) {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    void* ks = ws + wl.kshift_off;
    void* means = ws + wl.means_off;
    if (fp8_mode(mode)) kscale = reinterpret_cast<float*>(ws + wl.kscale_off);
    rc = kshift_dispatch(k, ks, means, kscale, B, Hkv, Sk, D, mode, st);
    if (rc != PASA_OK) return rc;
    kk = ks;
    mm = means;
  }
  return attn_launch(q, kk, mm, v, o, lse, B, Hq, Hkv, Sq, Sk, D, causal, scale, mode, st, nullptr, nullptr, kscale,
                     prep);
}

int pasa_attn_fwd_stats(const void* q, const void* k, const void* v, void* o, float* lse, float* stats,
                        float* block_stats, int B, int Hq, int Hkv, int Sq, int Sk, int D, int causal, float scale,
                        int mode, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = validate(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, D, mode);
  if (rc != PASA_OK) return rc;
  if (!stats) return PASA_ERR_NULLPTR;
  if ((reinterpret_cast<uintptr_t>(stats) & 7u) != 0) return PASA_ERR_ALIGN;
  if (block_stats && (reinterpret_cast<uintptr_t>(block_stats) & 7u) != 0) return PASA_ERR_ALIGN;
  if (fp8_mode(mode)) return PASA_ERR_UNSUPPORTED;  // no diagnostic build of the FP8 kernels
  const bool shift = shift_mode(mode);
  const WorkspaceLayout wl = workspace_layout(B, Hkv, Sk, D, mode);
  if (shift) {
    if (!workspace || workspace_bytes < wl.total) return PASA_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return PASA_ERR_ALIGN;
    if (static_cast<long long>(B) * Hkv > 65535) return PASA_ERR_SHAPE;
  }
  rc = check_device();
  if (rc != PASA_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const void* kk = k;
  const void* mm = k;
  if (shift) {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    rc = kshift_dispatch(k, ws + wl.kshift_off, ws + wl.means_off, nullptr, B, Hkv, Sk, D, mode, st);
    if (rc != PASA_OK) return rc;
    kk = ws + wl.kshift_off;
    mm = ws + wl.means_off;
  }
  return attn_launch(q, kk, mm, v, o, lse, B, Hq, Hkv, Sq, Sk, D, causal, scale, mode, st, stats, block_stats);
}

int pasa_attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv,
                  int Sq, int Sk, int D, int causal, float scale, int mode, void* stream) {
  int rc = validate(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, D, mode);
  if (rc != PASA_OK) return rc;
  const size_t bytes = pasa_attn_fwd_workspace_bytes(B, Hkv, Sk, D, mode);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  void* ws = nullptr;
  if (bytes > 0) {
    rc = check_device();
    if (rc != PASA_OK) return rc;
    cudaError_t e = cudaMallocAsync(&ws, bytes, st);
    if (e != cudaSuccess) return cuda_fail(e);
  }
  rc = pasa_attn_fwd_ws(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, D, causal, scale, mode, ws, bytes, stream);
  if (ws) {
    cudaError_t e = cudaFreeAsync(ws, st);
    if (rc == PASA_OK && e != cudaSuccess) rc = cuda_fail(e);
  }
  return rc;
}

int pasa_attn_fwd_fused(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv,
                        int Sq, int Sk, int D, int causal, float scale, int mode, void* k_shifted_out,
                        void* means_out, void* stream) {
  int rc = validate(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, D, mode);
  if (rc != PASA_OK) return rc;
  if (D != 128) return PASA_ERR_UNSUPPORTED;
  if (mode != PASA_MODE_SHIFT_F16ACC && mode != PASA_MODE_SHIFT_F32ACC && mode != PASA_MODE_SHIFT_F16ALL)
    return PASA_ERR_UNSUPPORTED;
  if ((k_shifted_out && !aligned16(k_shifted_out)) || (means_out && !aligned16(means_out))) return PASA_ERR_ALIGN;
  rc = check_device();
  if (rc != PASA_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!(scale > 0.0f) || !std::isfinite(scale)) scale = 1.0f / std::sqrt(static_cast<float>(D));
  const int bn = pasa::block_rows_for(D);
  CUtensorMap mq, mk, mv, mo;
  if ((rc = make_map(&mq, q, D, Sq, static_cast<long long>(B) * Hq, pasa::kTileRows)) != PASA_OK) return rc;
  if ((rc = make_map(&mk, k, D, Sk, static_cast<long long>(B) * Hkv, bn)) != PASA_OK) return rc;
  if ((rc = make_map(&mv, v, D, Sk, static_cast<long long>(B) * Hkv, bn)) != PASA_OK) return rc;
  if ((rc = make_map(&mo, o, D, Sq, static_cast<long long>(B) * Hq, pasa::kTileRows)) != PASA_OK) return rc;
  pasa::AttnParams p = {};
  p.lse = lse;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.Sq = Sq;
  p.Sk = Sk;
  p.n_qblk = (Sq + pasa::kTileRows - 1) / pasa::kTileRows;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.inv_scale_log2 = 1.0f / p.scale_log2;
  p.nbt = (Sk + bn - 1) / bn;
  p.sq_mod = Sq;
  p.kshift_out = static_cast<__half*>(k_shifted_out);
  p.means_out = static_cast<__half*>(means_out);
  switch (mode) {
    case PASA_MODE_SHIFT_F16ACC:
      return causal ? launch_attn_fused<true, true, false>(mq, mk, mv, mo, p, st)
                    : launch_attn_fused<true, false, false>(mq, mk, mv, mo, p, st);
    case PASA_MODE_SHIFT_F32ACC:
      return causal ? launch_attn_fused<false, true, false>(mq, mk, mv, mo, p, st)
                    : launch_attn_fused<false, false, false>(mq, mk, mv, mo, p, st);
    default:
      return causal ? launch_attn_fused<true, true, true>(mq, mk, mv, mo, p, st)
                    : launch_attn_fused<true, false, true>(mq, mk, mv, mo, p, st);
  }
}

int pasa_selftest_wait_timeout(void* stream) {
  int rc = check_device();
  if (rc != PASA_OK) return rc;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  rc = launch_wait_selftest(st, false);
  if (rc == PASA_OK) rc = pasa::packed_wait_selftest(st);
  if (rc == PASA_OK) rc = pasa::tree_wait_selftest(st);
  return rc;
}

int pasa_selftest_exp2(const float* x, float* poly, float* mufu, int n, void* stream) {
  if (!x || !poly || !mufu) return PASA_ERR_NULLPTR;
  if (n <= 0) return PASA_ERR_SHAPE;
  int rc = check_device();
  if (rc != PASA_OK) return rc;
  const int pairs = (n + 1) / 2;
  pasa::exp2_selftest_kernel<<<(pairs + 255) / 256, 256, 0, static_cast<cudaStream_t>(stream)>>>(x, poly, mufu, n);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? PASA_OK : cuda_fail(e);
}

int pasa_check_device_error(void* stream, unsigned long long* info) {
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e);
  // every translation unit has a record of its own: all are read and cleared, and the earliest timeout is reported
  int result = PASA_OK;
  unsigned long long first = ULLONG_MAX;
  for (int (*take)(pasa::DeviceError*) : {take_device_error, pasa::packed_take_device_error, pasa::tree_take_device_error}) {
    pasa::DeviceError found;
    const int rc = take(&found);
    if (rc == PASA_ERR_CUDA) return rc;
    if (rc == PASA_OK || found.at >= first) continue;
    result = rc;
    first = found.at;
    if (info) *info = found.info;
  }
  return result;
}

}  // extern "C"

// ---------------------------------------------------------------------------------------
// Allocation-free variant of pasa_attn_fwd.
//
// Some callers may not call cudaMalloc at all: a process whose device memory is owned by a
// framework or server allocator that reserves the whole GPU up front, or a latency-bound
// loop where an allocation (and the synchronisation it can imply) is not allowed. For them
// the shifted keys and block means live in one file-scope device array instead of a
// workspace. The array is part of this library's device image, so every GPU that loads
// the library holds it until the process exits.
// ---------------------------------------------------------------------------------------
#include <mutex>

namespace {

constexpr size_t kNoAllocScratchBytes = size_t(64) << 20;  // 64 MiB
static __device__ __align__(256) unsigned char g_noalloc_scratch[kNoAllocScratchBytes];

constexpr int kNoAllocMaxDevices = 64;
std::mutex g_noalloc_mutex;
void* g_noalloc_ptr[kNoAllocMaxDevices] = {};

// Device address of g_noalloc_scratch on the current device. The host-side name of the
// array is only a stand-in, so the address is looked up once per device (with that device
// current) and cached.
int noalloc_scratch(void** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev < 0 || dev >= kNoAllocMaxDevices) return PASA_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lock(g_noalloc_mutex);
  if (g_noalloc_ptr[dev] == nullptr) {
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_noalloc_scratch);
    if (e != cudaSuccess) return cuda_fail(e);
    g_noalloc_ptr[dev] = p;
  }
  *out = g_noalloc_ptr[dev];
  return PASA_OK;
}

}  // namespace

extern "C" int pasa_attn_fwd_noalloc(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                                     int Hq, int Hkv, int Sq, int Sk, int D, int causal, float scale, int mode,
                                     void* stream) {
  int rc = validate(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, D, mode);
  if (rc != PASA_OK) return rc;
  const size_t need = pasa_attn_fwd_workspace_bytes(B, Hkv, Sk, D, mode);
  if (need > kNoAllocScratchBytes) return PASA_ERR_WORKSPACE;
  rc = check_device();
  if (rc != PASA_OK) return rc;
  void* ws = nullptr;
  if (need > 0) {
    rc = noalloc_scratch(&ws);
    if (rc != PASA_OK) return rc;
  }
  return pasa_attn_fwd_ws(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, D, causal, scale, mode, ws,
                          need > 0 ? kNoAllocScratchBytes : 0, stream);
}

// ---------------------------------------------------------------------------------------
// Host-buffer forward: q, k, v in host memory, o and lse back to host memory, with the
// copies overlapped with the attention kernels.
//
// The (batch, kv head) pairs are the units of work: a unit's query heads, keys, values and
// outputs are contiguous in the [B, H, S, D] layouts, and a run of consecutive units is
// itself a problem of n units with one kv head, n standing in for B. The work is cut into
// pieces; piece i's host->device copies run on one side stream, its shift and attention
// kernels on the caller's stream once they have landed, and its device->host copies on a
// second side stream once they have finished. Copy engines and SMs then work at the same
// time, and only the first piece's inputs and the last piece's outputs are not hidden
// behind computation.
//
// To keep those two small, the automatic plan also cuts the first and the last unit along
// the query rows, in pieces that halve towards the ends ([0, Sq/8), [Sq/8, Sq/4),
// [Sq/4, Sq/2), ... for the first unit, mirrored for the last). A row piece [r0, r1) is the
// problem with Sq' = r1 - r0 query rows and, under the causal mask, the key prefix
// Sk' = r1 + Sk - Sq it can see: row r0 + i' sees key j iff j <= i' + Sk' - Sq', the same
// keys as before. With r0 on a 128-row tile boundary and Sk' on a 128-key block boundary
// (or Sk' = Sk) every query tile meets the same key blocks with the same pseudo-averages,
// so the results stay bit-identical to the single call. The unit's keys are copied once,
// in the slices each row piece adds.
// ---------------------------------------------------------------------------------------
#include <vector>

namespace {

constexpr int kHostMaxChunks = 64;
constexpr long long kHostMinChunkTiles = 256;  // query tiles of 128 rows a unit chunk keeps
constexpr long long kHostMinRowTiles = 128;    // ... and the smallest row piece keeps
constexpr int kHostMaxHalvings = 3;

struct HostPiece {
  int u0 = 0, n = 0;    // units [u0, u0 + n)
  int r0 = 0, r1 = 0;   // query rows [r0, r1) of each unit
  int k0 = 0, k1 = 0;   // keys this piece copies in; it attends keys [0, k1)
  bool rowcut = false;  // one of the query-row pieces of a unit
  size_t q_off = 0, kv_off = 0, o_off = 0, lse_off = 0;  // slots in the device buffer
  size_t prep_off = 0;  // rowcut with a key preparation: the unit's prepared keys (all Sk rows)
};

struct HostPlan {
  std::vector<HostPiece> pieces;
  int max_units = 0;  // units in the largest piece that is not a row piece
  size_t ws_off = 0, ws_bytes = 0, total = 0;
};

// Row boundaries for one unit: halving pieces at the front and/or the back, on 128-row
// tiles, the smallest with at least kHostMinRowTiles tiles over the unit's g heads.
std::vector<int> host_row_cuts(int Sq, int g, bool front, bool back) {
  std::vector<int> cuts{0};
  int halvings = 0;
  while (halvings < kHostMaxHalvings) {
    const long long rows = (static_cast<long long>(Sq) >> (halvings + 1)) / 128 * 128;
    if (rows <= 0 || static_cast<long long>(g) * (rows / 128) < kHostMinRowTiles) break;
    ++halvings;
  }
  if (halvings == 0 || (!front && !back)) {
    cuts.push_back(Sq);
    return cuts;
  }
  auto tile = [](long long r) { return static_cast<int>(r / 128 * 128); };
  if (front)
    for (int h = halvings; h >= 1; --h) cuts.push_back(tile(static_cast<long long>(Sq) >> h));
  else
    cuts.push_back(tile(static_cast<long long>(Sq) >> 1));
  if (back)
    for (int h = 2; h <= halvings; ++h) cuts.push_back(tile(Sq - (static_cast<long long>(Sq) >> h)));
  cuts.push_back(Sq);
  std::vector<int> out{0};
  for (size_t i = 1; i < cuts.size(); ++i)
    if (cuts[i] > out.back()) out.push_back(cuts[i]);
  return out;
}

// Pieces: the units cut into chunks (the requested count clamped to [1, min(units, 64)];
// 0 asks for as many as keep every chunk at >= 256 query tiles, at most 8). Only the
// automatic plan cuts the first and last unit into row pieces, and only where the row
// pieces keep the computation tile-for-tile the same (see above).
HostPlan host_plan(int B, int Hq, int Hkv, int Sq, int Sk, int D, int causal, int mode, int chunks) {
  HostPlan hp;
  const int units = B * Hkv;
  const int g = Hq / Hkv;
  const int cap = units < kHostMaxChunks ? units : kHostMaxChunks;
  const bool automatic = chunks <= 0;
  if (automatic) {
    const long long tiles = static_cast<long long>(g) * ((static_cast<long long>(Sq) + 127) / 128);
    int c = cap < 8 ? cap : 8;
    while (c > 1 && (units / c) * tiles < kHostMinChunkTiles) --c;
    chunks = c;
  }
  chunks = chunks < cap ? chunks : cap;
  const bool rows_ok = automatic && (!causal || (Sk >= Sq && (Sk - Sq) % 128 == 0));
  for (int c = 0; c < chunks; ++c) {
    const int a = static_cast<int>(static_cast<long long>(c) * units / chunks);
    const int b = static_cast<int>(static_cast<long long>(c + 1) * units / chunks);
    for (int u = a; u < b;) {
      const bool first = u == 0, last = u == units - 1;
      std::vector<int> cuts{0, Sq};
      if (rows_ok && (first || last)) cuts = host_row_cuts(Sq, g, first, last);
      if (cuts.size() > 2) {
        int kprev = 0;
        for (size_t i = 0; i + 1 < cuts.size(); ++i) {
          HostPiece pc;
          pc.u0 = u, pc.n = 1, pc.r0 = cuts[i], pc.r1 = cuts[i + 1], pc.rowcut = true;
          pc.k1 = causal ? pc.r1 + (Sk - Sq) : Sk;
          pc.k0 = kprev;
          kprev = pc.k1;
          hp.pieces.push_back(pc);
        }
        ++u;
        continue;
      }
      // a run of whole units up to the chunk's end or the next unit that is cut into rows
      int e = u + 1;
      while (e < b && !(rows_ok && e == units - 1 && host_row_cuts(Sq, g, false, true).size() > 2)) ++e;
      HostPiece pc;
      pc.u0 = u, pc.n = e - u, pc.r0 = 0, pc.r1 = Sq, pc.k0 = 0, pc.k1 = Sk;
      hp.pieces.push_back(pc);
      u = e;
    }
  }
  // slots: q and o [n, g, rows, D], lse [n, g, rows], and the keys/values [n, Sk, D] of a
  // unit once (row pieces after the first of a unit reuse it), with, for a unit cut into
  // row pieces, its prepared keys (shifted keys and means, or e4m3 codes and scales, for
  // all Sk rows): each row piece prepares only the key blocks it newly sees, the blocks
  // before them being final once written (a block's preparation reads that block only);
  // each slot 256-byte aligned
  const size_t row_bytes = static_cast<size_t>(D) * 2;
  const size_t prep_bytes = align_up(pasa_attn_fwd_workspace_bytes(1, 1, Sk, D, mode), 256);
  size_t off = 0, kv_last = 0, prep_last = 0;
  int kv_unit = -1;
  for (HostPiece& pc : hp.pieces) {
    const size_t nrows = static_cast<size_t>(pc.n) * g * (pc.r1 - pc.r0);
    pc.q_off = off;   off += align_up(nrows * row_bytes, 256);
    pc.o_off = off;   off += align_up(nrows * row_bytes, 256);
    pc.lse_off = off; off += align_up(nrows * 4, 256);
    if (pc.n == 1 && pc.k0 > 0 && kv_unit == pc.u0) {
      pc.kv_off = kv_last;
      pc.prep_off = prep_last;
    } else {
      pc.kv_off = kv_last = off;
      kv_unit = pc.n == 1 ? pc.u0 : -1;
      off += 2 * align_up(static_cast<size_t>(pc.n) * Sk * row_bytes, 256);
      if (pc.rowcut && prep_bytes > 0) {
        pc.prep_off = prep_last = off;
        off += prep_bytes;
      }
    }
    if (!pc.rowcut && pc.n > hp.max_units) hp.max_units = pc.n;
  }
  // one shift workspace per compute stream (pieces alternate between two), for the pieces of
  // whole units
  hp.ws_off = off;
  hp.ws_bytes = hp.max_units > 0 ? align_up(pasa_attn_fwd_workspace_bytes(hp.max_units, 1, Sk, D, mode), 256) : 0;
  hp.total = off + (hp.pieces.size() > 1 ? 2 : 1) * hp.ws_bytes;
  return hp;
}

// Three non-blocking side streams per device (host->device copies, device->host copies, a
// second compute stream), created on first use and kept for the life of the process. Calls
// from several host threads may share them: every wait a call enqueues refers to work that
// call has already enqueued, so the order stays acyclic.
std::mutex g_side_mutex;
cudaStream_t g_side_streams[kNoAllocMaxDevices][3] = {};

int side_streams(cudaStream_t* out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev < 0 || dev >= kNoAllocMaxDevices) return PASA_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lock(g_side_mutex);
  for (int j = 0; j < 3; ++j) {
    if (g_side_streams[dev][j] == nullptr) {
      e = cudaStreamCreateWithFlags(&g_side_streams[dev][j], cudaStreamNonBlocking);
      if (e != cudaSuccess) return cuda_fail(e);
    }
    out[j] = g_side_streams[dev][j];
  }
  return PASA_OK;
}

// `height` rows of `width` bytes between pitched buffers; one plain copy when both sides
// are contiguous.
cudaError_t copy_rows(void* dst, size_t dpitch, const void* src, size_t spitch, size_t width, size_t height,
                      cudaMemcpyKind kind, cudaStream_t st) {
  if (width == 0 || height == 0) return cudaSuccess;
  if (dpitch == width && spitch == width) return cudaMemcpyAsync(dst, src, width * height, kind, st);
  return cudaMemcpy2DAsync(dst, dpitch, src, spitch, width, height, kind, st);
}

}  // namespace

extern "C" int pasa_release_host_streams(void) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev < 0 || dev >= kNoAllocMaxDevices) return PASA_OK;   // none were ever created there
  std::lock_guard<std::mutex> lock(g_side_mutex);
  cudaError_t first = cudaSuccess;
  for (int j = 0; j < 3; ++j) {
    cudaStream_t& st = g_side_streams[dev][j];
    if (st == nullptr) continue;
    e = cudaStreamSynchronize(st);
    if (e == cudaSuccess) e = cudaStreamDestroy(st);
    if (e != cudaSuccess && first == cudaSuccess) first = e;
    st = nullptr;   // a failed destroy leaves the handle to the runtime; never reuse it
  }
  return first == cudaSuccess ? PASA_OK : cuda_fail(first);
}

extern "C" size_t pasa_attn_fwd_host_device_bytes(int B, int Hq, int Hkv, int Sq, int Sk, int D, int causal,
                                                   int mode, int chunks) {
  if (chunks < 0 || validate_shape(B, Hq, Hkv, Sq, Sk, D, mode) != PASA_OK) return 0;
  return host_plan(B, Hq, Hkv, Sq, Sk, D, causal, mode, chunks).total;
}

extern "C" int pasa_attn_fwd_host_plan(int B, int Hq, int Hkv, int Sq, int Sk, int D, int causal, int mode,
                                       int chunks, int* pieces, int max_pieces) {
  if (chunks < 0 || max_pieces < 0 || (max_pieces > 0 && !pieces)) return chunks < 0 ? PASA_ERR_SHAPE : PASA_ERR_NULLPTR;
  const int rc = validate_shape(B, Hq, Hkv, Sq, Sk, D, mode);
  if (rc != PASA_OK) return rc;
  const HostPlan hp = host_plan(B, Hq, Hkv, Sq, Sk, D, causal, mode, chunks);
  const int np = static_cast<int>(hp.pieces.size());
  for (int i = 0; i < np && i < max_pieces; ++i) {
    const HostPiece& pc = hp.pieces[i];
    int* r = pieces + 6 * static_cast<size_t>(i);
    r[0] = pc.u0, r[1] = pc.n, r[2] = pc.r0, r[3] = pc.r1, r[4] = pc.k0, r[5] = pc.k1;
  }
  return np;
}

extern "C" int pasa_attn_fwd_host(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq,
                                  int Hkv, int Sq, int Sk, int D, int causal, float scale, int mode, int chunks,
                                  void* device_buffer, size_t device_buffer_bytes, void* stream) {
  if (!q || !k || !v || !o) return PASA_ERR_NULLPTR;
  int rc = validate_shape(B, Hq, Hkv, Sq, Sk, D, mode);
  if (rc != PASA_OK) return rc;
  if (chunks < 0) return PASA_ERR_SHAPE;
  const HostPlan hp = host_plan(B, Hq, Hkv, Sq, Sk, D, causal, mode, chunks);
  if (device_buffer) {
    if (device_buffer_bytes < hp.total) return PASA_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(device_buffer) & 255u) != 0) return PASA_ERR_ALIGN;
  }
  rc = check_device();
  if (rc != PASA_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaStream_t side[3] = {};
  rc = side_streams(side);
  if (rc != PASA_OK) return rc;
  cudaStream_t s_in = side[0], s_out = side[1];
  cudaStream_t s_run[2] = {st, side[2]};  // piece i computes on s_run[i % 2]

  // events: [0] start on st, [1] h2d stream done, [2] d2h stream done, [3] second compute
  // stream done, [4 + i] piece i's inputs landed, [4 + np + i] piece i's kernels finished,
  // [4 + 2 np + i] a row piece's key blocks, and those of its unit's earlier pieces, prepared
  const int np = static_cast<int>(hp.pieces.size());
  std::vector<cudaEvent_t> ev(4 + 3 * static_cast<size_t>(np), nullptr);
  cudaError_t e = cudaSuccess;
  size_t made = 0;
  for (; made < ev.size(); ++made) {
    e = cudaEventCreateWithFlags(&ev[made], cudaEventDisableTiming);
    if (e != cudaSuccess) break;
  }
  uint8_t* buf = static_cast<uint8_t*>(device_buffer);
  bool owned = false;
  if (e == cudaSuccess && !buf) {
    e = cudaMallocAsync(reinterpret_cast<void**>(&buf), hp.total, st);
    owned = e == cudaSuccess;
  }
  if (e != cudaSuccess) {
    for (size_t j = 0; j < made; ++j) cudaEventDestroy(ev[j]);
    return cuda_fail(e);
  }

  // Everything below is enqueued on st, s_in or s_out; on the first failure the rest is
  // skipped, but the side streams are still joined back to st before the buffer is freed.
  auto step = [&](cudaError_t err) {
    if (e == cudaSuccess && err != cudaSuccess) e = err;
    return e == cudaSuccess;
  };
  const int g = Hq / Hkv;
  const size_t row_bytes = static_cast<size_t>(D) * 2;
  const size_t q_unit = static_cast<size_t>(g) * Sq * row_bytes;  // bytes of one unit's q (and o)
  const size_t kv_unit = static_cast<size_t>(Sk) * row_bytes;
  const size_t lse_unit = static_cast<size_t>(g) * Sq * 4;
  const uint8_t* qh = static_cast<const uint8_t*>(q);
  const uint8_t* kh = static_cast<const uint8_t*>(k);
  const uint8_t* vh = static_cast<const uint8_t*>(v);
  uint8_t* oh = static_cast<uint8_t*>(o);
  uint8_t* lh = reinterpret_cast<uint8_t*>(lse);

  // the buffer may still be in use by work the caller queued on st before this call
  step(cudaEventRecord(ev[0], st));
  step(cudaStreamWaitEvent(s_in, ev[0], 0));
  step(cudaStreamWaitEvent(s_out, ev[0], 0));
  step(cudaStreamWaitEvent(s_run[1], ev[0], 0));
  for (int i = 0; i < np && e == cudaSuccess; ++i) {
    const HostPiece& pc = hp.pieces[i];
    const size_t kv_bytes = align_up(static_cast<size_t>(pc.n) * kv_unit, 256);
    uint8_t* kd = buf + pc.kv_off;
    uint8_t* vd = kd + kv_bytes;
    // whole units: all their keys; a row piece: the keys [k0, k1) its rows newly see
    const size_t kb0 = static_cast<size_t>(pc.k0) * row_bytes;
    const size_t nb = pc.n == 1 ? static_cast<size_t>(pc.k1 - pc.k0) * row_bytes : pc.n * kv_unit;
    step(copy_rows(kd + kb0, nb, kh + pc.u0 * kv_unit + kb0, nb, nb, 1, cudaMemcpyHostToDevice, s_in));
    step(copy_rows(vd + kb0, nb, vh + pc.u0 * kv_unit + kb0, nb, nb, 1, cudaMemcpyHostToDevice, s_in));
    const size_t w = static_cast<size_t>(pc.r1 - pc.r0) * row_bytes;
    step(copy_rows(buf + pc.q_off, w, qh + pc.u0 * q_unit + pc.r0 * row_bytes, static_cast<size_t>(Sq) * row_bytes,
                   w, static_cast<size_t>(pc.n) * g, cudaMemcpyHostToDevice, s_in));
    step(cudaEventRecord(ev[4 + i], s_in));
  }
  const bool prep = shift_mode(mode) || fp8_mode(mode);
  const WorkspaceLayout pl = workspace_layout(1, 1, Sk, D, mode);   // a row-cut unit's prepared keys
  const int bn = pasa::block_rows_for(D);
  for (int i = 0; i < np && e == cudaSuccess; ++i) {
    const HostPiece& pc = hp.pieces[i];
    const size_t kv_bytes = align_up(static_cast<size_t>(pc.n) * kv_unit, 256);
    const int rows = pc.r1 - pc.r0;
    cudaStream_t run = s_run[i & 1];
    if (!step(cudaStreamWaitEvent(run, ev[4 + i], 0))) break;
    int krc = PASA_OK;
    if (pc.rowcut && prep) {
      // prepare this piece's new key blocks [k0, k1) into the unit's slot, then wait until
      // the unit's earlier pieces have prepared theirs (on either compute stream)
      uint8_t* pb = buf + pc.prep_off;
      float* kscale = fp8_mode(mode) ? reinterpret_cast<float*>(pb + pl.kscale_off) : nullptr;
      if (pc.k1 > pc.k0) krc = kshift_dispatch(buf + pc.kv_off, pb + pl.kshift_off, pb + pl.means_off, kscale, 1, 1,
                                               pc.k1, D, mode, run, pc.k0 / bn, Sk);
      if (krc == PASA_OK && i > 0 && hp.pieces[i - 1].rowcut && hp.pieces[i - 1].u0 == pc.u0)
        step(cudaStreamWaitEvent(run, ev[4 + 2 * np + i - 1], 0));
      step(cudaEventRecord(ev[4 + 2 * np + i], run));
      if (krc == PASA_OK && e == cudaSuccess)
        krc = attn_launch(buf + pc.q_off, pb + pl.kshift_off, pb + pl.means_off, buf + pc.kv_off + kv_bytes,
                          buf + pc.o_off, lse ? reinterpret_cast<float*>(buf + pc.lse_off) : nullptr, 1, g, 1, rows,
                          pc.k1, D, causal, scale, mode, run, nullptr, nullptr, kscale);
    } else {
      krc = pasa_attn_fwd_ws(buf + pc.q_off, buf + pc.kv_off, buf + pc.kv_off + kv_bytes, buf + pc.o_off,
                             lse ? reinterpret_cast<float*>(buf + pc.lse_off) : nullptr, pc.n, g, 1, rows, pc.k1, D,
                             causal, scale, mode, hp.ws_bytes ? buf + hp.ws_off + (i & 1) * hp.ws_bytes : nullptr,
                             hp.ws_bytes, run);
    }
    if (krc != PASA_OK) {
      rc = krc;
      break;
    }
    step(cudaEventRecord(ev[4 + np + i], run));
    step(cudaStreamWaitEvent(s_out, ev[4 + np + i], 0));
    const size_t w = static_cast<size_t>(rows) * row_bytes;
    const size_t h = static_cast<size_t>(pc.n) * g;
    step(copy_rows(oh + pc.u0 * q_unit + pc.r0 * row_bytes, static_cast<size_t>(Sq) * row_bytes, buf + pc.o_off, w,
                   w, h, cudaMemcpyDeviceToHost, s_out));
    if (lse)
      step(copy_rows(lh + pc.u0 * lse_unit + static_cast<size_t>(pc.r0) * 4, static_cast<size_t>(Sq) * 4,
                     buf + pc.lse_off, static_cast<size_t>(rows) * 4, static_cast<size_t>(rows) * 4, h,
                     cudaMemcpyDeviceToHost, s_out));
  }
  // join: st continues only after the side streams have drained this call's work
  cudaError_t je = cudaSuccess;
  for (int j = 0; j < 3 && je == cudaSuccess; ++j) {
    je = cudaEventRecord(ev[1 + j], side[j]);
    if (je == cudaSuccess) je = cudaStreamWaitEvent(st, ev[1 + j], 0);
  }
  if (je != cudaSuccess) {
    // st cannot be ordered after the side streams: wait for them here before freeing
    for (int j = 0; j < 3; ++j) cudaStreamSynchronize(side[j]);
    step(je);
  }
  if (owned) step(cudaFreeAsync(buf, st));
  for (cudaEvent_t x : ev) cudaEventDestroy(x);
  if (rc != PASA_OK) return rc;
  return e == cudaSuccess ? PASA_OK : cuda_fail(e);
}

// ---------------------------------------------------------------------------------------
// 4-bit key/value cache
// ---------------------------------------------------------------------------------------
namespace {

// kv4_append and kv4_read share their arguments: n rows of k and v from cache row `start` on.
int kv4_window(const void* k, const void* v, const int* starts, int start, const int* counts, int n, int B, int Hkv,
               int Sk_cap, int D, bool append, pasa::Kv4Window* win, dim3* grid) {
  if (!k || !v) return PASA_ERR_NULLPTR;
  if (n <= 0) return PASA_ERR_SHAPE;
  if (!starts && (start < 0 || static_cast<long long>(start) + n > Sk_cap)) return PASA_ERR_SHAPE;
  if (!aligned16(k) || !aligned16(v) || !aligned4(starts) || !aligned4(counts)) return PASA_ERR_ALIGN;
  if (n > INT_MAX - 256) return PASA_ERR_SHAPE;   // row numbers of a block's last threads
  const int per_block = append ? pasa::kKv4AppendRows * (pasa::kKv4StoreThreads / (D / 16)) : pasa::kKv4ReadRows * (pasa::kKv4StoreThreads / (D / 8));
  *win = pasa::Kv4Window{starts, counts, start, n, Sk_cap};
  *grid = dim3(static_cast<unsigned>((n + per_block - 1) / per_block), static_cast<unsigned>(std::min(B * Hkv, 65535)));
  return PASA_OK;
}

// How a decode call is laid out: query rows in tiles of 8 (NT = 1) or 16, and either a cluster of CTAs per
// (sequence, kv head, row tile), or a fixed number of CTAs sharing all their keys evenly with
// partial results in the workspace. The numbers of CTAs and clusters (here, in kv4_ctas and in the eviction's
// clusters) are those of GB300's 152 SMs: right on any number, chosen for that one.
constexpr int kKv4MaxKeys = INT_MAX - 65536;   // key numbers past the last unit's fit an int

struct Kv4Plan {
  int nt, row_tiles, ctas, cluster;
  bool stream_k;
  long long segments;
  size_t part_o, part_ml, lse2, total;   // workspace: byte offsets and size
};

// Query rows of a tile.
int kv4_tile(int rows) { return rows <= 8 ? 8 : 16; }

// Whether a call's segments, each of its rounds and the weight of its start, fit an int: grids and shares are
// ints. rows <= kTileRows, Sk <= kKv4MaxKeys. To be asked before kv4_plan.
bool kv4_fits(int B, int Hkv, int rows, int Sk) {
  const long long heads = static_cast<long long>(B) * Hkv;
  const int units = (Sk + pasa::kKv4Unit - 1) / pasa::kKv4Unit, tile = kv4_tile(rows);
  return heads <= INT_MAX && heads * ((rows + tile - 1) / tile) <= INT_MAX / (units + pasa::kKv4SegmentStart);
}

Kv4Plan kv4_plan(int B, int Hq, int Hkv, int Sq, int Sk, int D, bool weights) {
  Kv4Plan pl = {};
  const int rows = Hq / Hkv * Sq;
  pl.nt = kv4_tile(rows) / 8;
  pl.row_tiles = (rows + 8 * pl.nt - 1) / (8 * pl.nt);
  pl.segments = static_cast<long long>(B) * Hkv * pl.row_tiles;
  pl.ctas = pasa::kv4_ctas(pl.nt);
  const int units = (Sk + pasa::kKv4Unit - 1) / pasa::kKv4Unit;
  const int warps = pasa::kv4_warps(pl.nt);
  // A cluster per segment: as many CTAs as find an SM each while all clusters run at once, but no more than
  // take a round of their warps off. Clusters of c CTAs on 152 SMs (occupancy query; each stays
  // within a GPC): one past the number costs a second wave (16 segments of 56 rows x 8192 keys: 14.1 us
  // with 6 CTAs, 20.9 with 8), two CTAs on an SM about as much (16 of 7 rows x 4096 keys: 8.2 with 6, 9.6 with 8).
  constexpr int kClusters[9] = {0, INT_MAX, 76, 46, 36, 28, 23, 15, 15};
  int most = 8;
  while (most > 1 && pl.segments > kClusters[most]) --most;
  const int rounds = (units + warps * most - 1) / (warps * most);
  pl.cluster = (units + warps * rounds - 1) / (warps * rounds);
  // That needs one launch and no workspace, but few segments leave SMs idle, and an uneven batch
  // waits for its longest sequence. GPU us with D = 128, cluster against stream-K, whose launches cost the host
  // 8 us more, by segments x CTAs and rounds; 7 rows: 4 x 8 (6) 11.2 / 9.7, 8 x 8 (6) 11.3 / 11.3, 16 x 6 (8)
  // 13.8 / 14.5, 96 x 1 (16) 21.1 / 20.4, 32 x 4 (16) 22.4 / 22.2, (24) 30.8 / 28.2, 64 x 2 (16) 22.5 / 22.6, (32) 39.1 /
  // 35.1, 152 x 1 (16) 21.6 / 30.2; 16-row tiles: 8 x 8 (4) 14.3 / 12.7, 16 x 6 (6) 17.8 / 16.7, 28 x 5 (13) 30.1 / 33.4,
  // 40 x 3 (15) 33.0 / 33.6, 112 x 1 (11) 24.8 / 32.4, 200 x 1 (22) 84.5 / 76.2.
  const long long filled = pl.segments * most * 100 / 152;   // percent of the SMs
  pl.stream_k = rounds > (filled < 50 ? 6 : filled < 70 ? 8 : 16);
  if (pl.stream_k) pl.cluster = 1;
  const size_t tile = static_cast<size_t>(8 * pl.nt);
  const size_t slots = pl.stream_k ? static_cast<size_t>(2 * pl.ctas) : 0;
  pl.part_o = 0;
  pl.part_ml = align_up(slots * tile * D * 4, 256);
  pl.lse2 = pl.part_ml + align_up(slots * tile * 8, 256);
  pl.total = pl.lse2 + (weights ? align_up(static_cast<size_t>(pl.segments) * tile * 4, 256) : 0);
  return pl;
}

template <int D, int NT, bool STREAM_K>
cudaError_t kv4_launch(const pasa::Kv4Params& p, unsigned grid, cudaStream_t st, bool pdl) {
  static std::atomic<unsigned long long> raised{0};
  constexpr int need = static_cast<int>(sizeof(pasa::Kv4Smem<D, NT>)), most = std::max(need, pasa::kKv4Alone);
  // In a step (pdl) the clusters' CTAs start while the append's still hold SMs, and would go two to an SM elsewhere: where
  // there is an SM for each, it asks for one alone. GPU us of a step with 7 rows x 4 heads, two to an SM / alone / append and
  // decode as two calls: 8 x 4096 keys 14.6 / 11.0 / 11.9, 16 x 4096 22.6 / 15.7 / 16.6, 24 x 2048 21.4 / 14.7 / 15.5, 1 x 2048
  // 7.4 / 7.4 / 8.2, 512 new rows of 2 x 4096 11.0 / 8.8 / 9.7; with weights 8 x 4096 19.4 / 16.4, 6 x 4096 15.4 / 15.8.
  // The decode call by itself takes the same either way (8 x 4096: 9.2), but with weights, whose kernel
  // shares the SMs with it, longer alone (14.1 / 14.6).
  const int smem = pdl && !STREAM_K && grid <= pasa::kv4_ctas(2) ? most : need;
  return launch_clusters(pasa::kv4_decode_kernel<D, NT, STREAM_K>, grid, pasa::kv4_warps(NT) * 32, smem, most, st, pdl,
                         p.cluster, raised, p);
}

template <int D>
cudaError_t kv4_decode_launch(const pasa::Kv4Params& p, const Kv4Plan& pl, cudaStream_t st, bool pdl) {
  const unsigned grid = static_cast<unsigned>(pl.stream_k ? pl.ctas : pl.segments * pl.cluster);
  const int tile = 8 * pl.nt;
  cudaError_t e = pl.nt == 1 ? (pl.stream_k ? kv4_launch<D, 1, true>(p, grid, st, pdl) : kv4_launch<D, 1, false>(p, grid, st, pdl))
                             : (pl.stream_k ? kv4_launch<D, 2, true>(p, grid, st, pdl) : kv4_launch<D, 2, false>(p, grid, st, pdl));
  if (e == cudaSuccess && pl.stream_k)
    e = launch_kernel(pasa::kv4_merge_kernel<D>, dim3(static_cast<unsigned>(pl.segments), tile), dim3(256), 0, st, true,
                      p, tile);
  if (e == cudaSuccess && p.weights) {
    // Two CTAs per SM share the longest cases best. Where one to each SM is enough, two would pile up on the SMs
    // that the decode does not hold when they start; alone, a CTA has the registers to take both halves of a
    // unit side by side, which counts with more than 8 rows. GPU us of a call, two / alone, 4 heads: 112 rows x 1024 keys (24
    // rounds) 16.3 / 15.6, x 4096 (72) 23.6 / 20.1, x 8192 (136) 28.1 / 24.6, x 9600 (160) 28.2 / 28.3, x 16384 (264) 35.6 /
    // 36.0, x 131072 187 / 195; 56 rows x 8192 21.4 / 19.9; 28 rows x 8192 17.8 / 16.7, x 16384 23.6 / 23.6; 16 rows x 8192
    // 16.4 / 15.9; 9 rows x 1024 10.6 / 10.4; 7 rows x 2048 8.5 / 8.4, x 8192 12.5 / 12.7.
    const int all = pasa::kv4_ctas(1);
    int smem = static_cast<int>(offsetof(pasa::Kv4WeightsSmem<D>, q) + sizeof(pasa::Kv4QueryShared<D>) * ((p.rows + 7) / 8));
    const int rounds = pasa::kv4_rounds(pasa::kv4_units(p.Sk), pasa::kKv4WeightsWarps) + pasa::kKv4SegmentStart;
    const bool alone = p.rows > 8 && static_cast<long long>(p.B) * p.Hkv * rounds <= all / 2;
    if (alone) smem = std::max(smem, pasa::kKv4Alone);
    static std::atomic<unsigned long long> raised{0}, raised_alone{0};
    e = launch_clusters(alone ? pasa::kv4_weights_kernel<D, true> : pasa::kv4_weights_kernel<D, false>,
                        alone ? all / 2 : all, pasa::kKv4WeightsWarps * 32, smem, pasa::kKv4Alone, st, true, 1,
                        alone ? raised_alone : raised, p, tile);
  }
  return e;
}

}  // namespace

extern "C" {

// The checks of an append, and its launch. pick: the rows of k and v [B, Hkv, n_src, D] to store, or nullptr.
static int kv4_append_check(const void* k, const void* v, const void* shift, const void* k4, const void* kscale,
                            const void* v4, const void* vscale, const int* starts, int start, const int* counts, int B,
                            int Hkv, int n, int Sk_cap, int D, pasa::Kv4Window* win, dim3* grid,
                            const int* pick = nullptr, int n_src = 0) {
  int rc = kv4_validate(k4, kscale, v4, vscale, shift, B, Hkv, Sk_cap, D);
  if (rc != PASA_OK) return rc;
  rc = kv4_window(k, v, starts, start, counts, n, B, Hkv, Sk_cap, D, true, win, grid);
  if (rc != PASA_OK) return rc;
  const Kv4Spans c(k4, kscale, v4, vscale, shift, B, Hkv, Sk_cap, D);
  const unsigned long long rows = static_cast<unsigned long long>(B) * Hkv * (pick ? n_src : n);
  const bool shared = any_meet({c.k4, c.kscale, c.v4, c.vscale},
                               {Span(k, rows, 2 * D), Span(v, rows, 2 * D), c.shift, Span(starts, B, 4), Span(counts, B, 4),
                                Span(pick, static_cast<unsigned long long>(B) * n, 4)});
  return shared ? PASA_ERR_SHAPE : PASA_OK;
}

static int kv4_append_enqueue(const void* k, const void* v, const void* shift, void* k4, void* kscale, void* v4, void* vscale,
                              int B, int Hkv, int D, const pasa::Kv4Window& win, dim3 grid, cudaStream_t st,
                              const int* pick = nullptr, int n_src = 0) {
  auto kern = D == 64 ? (pick ? pasa::kv4_append_kernel<64, true> : pasa::kv4_append_kernel<64, false>)
                      : (pick ? pasa::kv4_append_kernel<128, true> : pasa::kv4_append_kernel<128, false>);
  kern<<<grid, pasa::kKv4StoreThreads, 0, st>>>(
      static_cast<const __half*>(k), static_cast<const __half*>(v), static_cast<const __half*>(shift),
      static_cast<uint8_t*>(k4), static_cast<__half*>(kscale), static_cast<uint8_t*>(v4), static_cast<__half*>(vscale),
      B * Hkv, Hkv, win, pick, n_src);
  return launch_status();
}

int pasa_kv4_append(const void* k, const void* v, const void* shift, void* k4, void* kscale, void* v4, void* vscale,
                    const int* starts, int start, const int* counts, int B, int Hkv, int n, int Sk_cap, int D,
                    void* stream) {
  pasa::Kv4Window win;
  dim3 grid;
  int rc = kv4_append_check(k, v, shift, k4, kscale, v4, vscale, starts, start, counts, B, Hkv, n, Sk_cap, D, &win, &grid);
  if (rc != PASA_OK) return rc;
  rc = check_device();
  if (rc != PASA_OK) return rc;
  return kv4_append_enqueue(k, v, shift, k4, kscale, v4, vscale, B, Hkv, D, win, grid, static_cast<cudaStream_t>(stream));
}

int pasa_kv4_append_rows(const void* k, const void* v, const void* shift, void* k4, void* kscale, void* v4, void* vscale,
                         const int* rows, const int* starts, int start, const int* counts, int B, int Hkv, int n, int n_src,
                         int Sk_cap, int D, void* stream) {
  if (!rows) return PASA_ERR_NULLPTR;
  if (n_src <= 0) return PASA_ERR_SHAPE;
  if (!aligned4(rows)) return PASA_ERR_ALIGN;
  pasa::Kv4Window win;
  dim3 grid;
  int rc = kv4_append_check(k, v, shift, k4, kscale, v4, vscale, starts, start, counts, B, Hkv, n, Sk_cap, D, &win, &grid,
                            rows, n_src);
  if (rc != PASA_OK) return rc;
  rc = check_device();
  if (rc != PASA_OK) return rc;
  return kv4_append_enqueue(k, v, shift, k4, kscale, v4, vscale, B, Hkv, D, win, grid, static_cast<cudaStream_t>(stream),
                            rows, n_src);
}

int pasa_kv4_read(const void* k4, const void* kscale, const void* v4, const void* vscale, const void* shift, void* k,
                  void* v, const int* starts, int start, const int* counts, int B, int Hkv, int n, int Sk_cap, int D,
                  void* stream) {
  int rc = kv4_validate(k4, kscale, v4, vscale, shift, B, Hkv, Sk_cap, D);
  if (rc != PASA_OK) return rc;
  pasa::Kv4Window win;
  dim3 grid;
  rc = kv4_window(k, v, starts, start, counts, n, B, Hkv, Sk_cap, D, false, &win, &grid);
  if (rc != PASA_OK) return rc;
  const Kv4Spans c(k4, kscale, v4, vscale, shift, B, Hkv, Sk_cap, D);
  const unsigned long long rows = static_cast<unsigned long long>(B) * Hkv * n;
  if (any_meet({Span(k, rows, 2 * D), Span(v, rows, 2 * D)},
               {c.k4, c.kscale, c.v4, c.vscale, c.shift, Span(starts, B, 4), Span(counts, B, 4)}))
    return PASA_ERR_SHAPE;
  rc = check_device();
  if (rc != PASA_OK) return rc;
  auto kern = D == 64 ? pasa::kv4_read_kernel<64> : pasa::kv4_read_kernel<128>;
  kern<<<grid, pasa::kKv4StoreThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint8_t*>(k4), static_cast<const __half*>(kscale), static_cast<const uint8_t*>(v4),
      static_cast<const __half*>(vscale), static_cast<const __half*>(shift), static_cast<__half*>(k),
      static_cast<__half*>(v), B * Hkv, Hkv, win);
  return launch_status();
}

size_t pasa_attn_fwd_decode_kv4_workspace_bytes(int B, int Hq, int Hkv, int Sq, int Sk, int D, int weights) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Sq <= 0 || Sk <= 0 || Hq % Hkv != 0 || Sk > kKv4MaxKeys || (D != 64 && D != 128))
    return 0;
  if (static_cast<long long>(Hq / Hkv) * Sq > pasa::kTileRows) return 0;
  if (!kv4_fits(B, Hkv, Hq / Hkv * Sq, Sk)) return 0;
  return kv4_plan(B, Hq, Hkv, Sq, Sk, D, weights != 0).total;
}

// The checks of a decode call, and its layout.
static int kv4_decode_check(const void* q, const void* k4, const void* kscale, const void* v4, const void* vscale,
                            const void* shift, const int* lengths, const void* o, const float* lse, const float* weights,
                            int B, int Hq, int Hkv, int Sq, int Sk, int Sk_cap, int D, const void* workspace,
                            size_t workspace_bytes, Kv4Plan* plan) {
  if (!q || !o) return PASA_ERR_NULLPTR;
  const int rc = kv4_validate(k4, kscale, v4, vscale, shift, B, Hkv, Sk_cap, D);
  if (rc != PASA_OK) return rc;
  if (Hq <= 0 || Sq <= 0 || Sk <= 0 || Hq % Hkv != 0 || Sk_cap < Sk || Sk > kKv4MaxKeys) return PASA_ERR_SHAPE;
  if (static_cast<long long>(Hq / Hkv) * Sq > pasa::kTileRows) return PASA_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(o) || !aligned16(lse) || !aligned16(weights) || !aligned4(lengths))
    return PASA_ERR_ALIGN;
  if (!kv4_fits(B, Hkv, Hq / Hkv * Sq, Sk)) return PASA_ERR_SHAPE;
  *plan = kv4_plan(B, Hq, Hkv, Sq, Sk, D, weights != nullptr);
  if (plan->total > 0) {
    if (!workspace || workspace_bytes < plan->total) return PASA_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return PASA_ERR_ALIGN;
  }
  return PASA_OK;
}

// Whether a decode call's outputs or workspace share memory with one another or with what it reads. Without
// `weights` o may be q itself: the kernel that writes a row of o is the last to read that row of q.
static bool kv4_decode_meets(const Kv4Plan& pl, const void* q, const void* k4, const void* kscale, const void* v4,
                             const void* vscale, const void* shift, const int* lengths, const void* o, const float* lse,
                             const float* weights, int B, int Hq, int Hkv, int Sq, int Sk_cap, int D, const void* workspace) {
  const Kv4Spans c(k4, kscale, v4, vscale, shift, B, Hkv, Sk_cap, D);
  const unsigned long long rows = static_cast<unsigned long long>(B) * Hq * Sq;
  const Span qs(q, rows, 2 * D), os(o, rows, 2 * D), ls(lse, rows, 4);
  const Span ws(weights, static_cast<unsigned long long>(B) * Hkv * Sk_cap, 4), work(pl.total ? workspace : nullptr, pl.total, 1);
  const Span lens(lengths, B, 4);
  return any_meet({os, ls, ws, work}, {c.k4, c.kscale, c.v4, c.vscale, c.shift, lens}) ||
         any_meet({ls, ws, work}, {qs}) || ((weights || o != q) && os.meets(qs));
}

// The kernels of a checked decode call. len_add: added to lengths[]; pdl: the kernel ahead on the
// stream is this call's append, which the decode waits for before it reads codes and scales.
static int kv4_decode_enqueue(const Kv4Plan& pl, const void* q, const void* k4, const void* kscale, const void* v4,
                              const void* vscale, const void* shift, const int* lengths, int len_add, void* o, float* lse,
                              float* weights, int B, int Hq, int Hkv, int Sq, int Sk, int Sk_cap, int D, int causal,
                              float scale, void* workspace, cudaStream_t st, bool pdl) {
  if (!(scale > 0.0f) || !std::isfinite(scale)) scale = 1.0f / std::sqrt(static_cast<float>(D));
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  pasa::Kv4Params p = {};
  p.q = static_cast<const __half*>(q);
  p.k4 = static_cast<const uint8_t*>(k4);
  p.v4 = static_cast<const uint8_t*>(v4);
  p.kscale = static_cast<const __half*>(kscale);
  p.vscale = static_cast<const __half*>(vscale);
  p.shift = static_cast<const __half*>(shift);
  p.lengths = lengths;
  p.len_add = len_add;
  p.o = static_cast<__half*>(o);
  p.lse = lse;
  p.weights = weights;
  p.part_o = reinterpret_cast<float*>(ws + pl.part_o);
  p.part_ml = reinterpret_cast<float2*>(ws + pl.part_ml);
  p.lse2 = reinterpret_cast<float*>(ws + pl.lse2);
  p.B = B;
  p.Hkv = Hkv;
  p.Sq = Sq;
  p.rows = Hq / Hkv * Sq;
  p.row_tiles = pl.row_tiles;
  p.Sk = Sk;
  p.cap = Sk_cap;
  p.causal = causal ? 1 : 0;
  p.ctas = pl.ctas;
  p.cluster = pl.cluster;
  p.scale = scale;
  p.scale_log2 = scale * 1.4426950408889634f;
  const cudaError_t e = D == 64 ? kv4_decode_launch<64>(p, pl, st, pdl) : kv4_decode_launch<128>(p, pl, st, pdl);
  return e == cudaSuccess ? launch_status() : cuda_fail(e);
}

int pasa_attn_fwd_decode_kv4(const void* q, const void* k4, const void* kscale, const void* v4, const void* vscale,
                             const void* shift, const int* lengths, void* o, float* lse, float* weights, int B, int Hq,
                             int Hkv, int Sq, int Sk, int Sk_cap, int D, int causal, float scale, void* workspace,
                             size_t workspace_bytes, void* stream) {
  Kv4Plan pl;
  int rc = kv4_decode_check(q, k4, kscale, v4, vscale, shift, lengths, o, lse, weights, B, Hq, Hkv, Sq, Sk, Sk_cap, D,
                            workspace, workspace_bytes, &pl);
  if (rc != PASA_OK) return rc;
  if (kv4_decode_meets(pl, q, k4, kscale, v4, vscale, shift, lengths, o, lse, weights, B, Hq, Hkv, Sq, Sk_cap, D, workspace))
    return PASA_ERR_SHAPE;
  rc = check_device();
  if (rc != PASA_OK) return rc;
  return kv4_decode_enqueue(pl, q, k4, kscale, v4, vscale, shift, lengths, 0, o, lse, weights, B, Hq, Hkv, Sq, Sk, Sk_cap,
                            D, causal, scale, workspace, static_cast<cudaStream_t>(stream), false);
}

int pasa_attn_fwd_decode_step_kv4(const void* q, const void* k, const void* v, void* k4, void* kscale, void* v4,
                                  void* vscale, const void* shift, const int* starts, int start, void* o, float* lse,
                                  float* weights, int B, int Hq, int Hkv, int Sq, int n, int Sk, int Sk_cap, int D,
                                  int causal, float scale, void* workspace, size_t workspace_bytes, void* stream) {
  if (n <= 0) return PASA_ERR_SHAPE;
  if (!starts) {   // every sequence has start + n rows in the end
    if (start < 0 || static_cast<long long>(start) + n > Sk_cap) return PASA_ERR_SHAPE;
    Sk = start + n;
  }
  Kv4Plan pl;
  int rc = kv4_decode_check(q, k4, kscale, v4, vscale, shift, starts, o, lse, weights, B, Hq, Hkv, Sq, Sk, Sk_cap, D,
                            workspace, workspace_bytes, &pl);
  if (rc != PASA_OK) return rc;
  pasa::Kv4Window win;
  dim3 grid;
  rc = kv4_append_check(k, v, shift, k4, kscale, v4, vscale, starts, start, nullptr, B, Hkv, n, Sk_cap, D, &win, &grid);
  if (rc != PASA_OK) return rc;
  const Kv4Spans c(k4, kscale, v4, vscale, shift, B, Hkv, Sk_cap, D);   // what the append writes, and q
  if (any_meet({c.k4, c.kscale, c.v4, c.vscale}, {Span(q, static_cast<unsigned long long>(B) * Hq * Sq, 2 * D)}))
    return PASA_ERR_SHAPE;
  if (kv4_decode_meets(pl, q, k4, kscale, v4, vscale, shift, starts, o, lse, weights, B, Hq, Hkv, Sq, Sk_cap, D, workspace))
    return PASA_ERR_SHAPE;
  rc = check_device();
  if (rc != PASA_OK) return rc;
  rc = kv4_append_enqueue(k, v, shift, k4, kscale, v4, vscale, B, Hkv, D, win, grid, static_cast<cudaStream_t>(stream));
  if (rc != PASA_OK) return rc;
  return kv4_decode_enqueue(pl, q, k4, kscale, v4, vscale, shift, starts, n, o, lse, weights, B, Hq, Hkv, Sq, Sk, Sk_cap, D,
                            causal, scale, workspace, static_cast<cudaStream_t>(stream), true);
}

int pasa_cache_evict(const void* const* planes, void* const* out_planes, const int* row_bytes, int n_planes,
                     const float* weights, float* out_weights, const int* lengths, int* index, int* new_lengths, int B,
                     int Hkv, int Sk, int Sk_cap, int out_cap, int budget, int recent, void* stream) {
  if (!planes || !out_planes || !row_bytes || !weights || !out_weights || !index) return PASA_ERR_NULLPTR;
  if (B <= 0 || Hkv <= 0 || Sk <= 0 || Sk_cap < Sk) return PASA_ERR_SHAPE;
  if (static_cast<long long>(B) * Hkv * pasa::kEvictCluster > INT_MAX) return PASA_ERR_SHAPE;
  if (budget <= 0 || recent < 0 || recent > budget || out_cap < budget) return PASA_ERR_SHAPE;
  if (n_planes < 1 || n_planes > pasa::kEvictPlanes) return PASA_ERR_UNSUPPORTED;
  if (!aligned16(weights) || !aligned16(out_weights) || !aligned16(index) || !aligned4(lengths) || !aligned4(new_lengths))
    return PASA_ERR_ALIGN;
  bool in_place = weights == out_weights, apart = !in_place;
  for (int i = 0; i < n_planes; ++i) {
    if (!planes[i] || !out_planes[i]) return PASA_ERR_NULLPTR;
    if (row_bytes[i] <= 0 || row_bytes[i] > 65536) return PASA_ERR_SHAPE;
    if (row_bytes[i] % 4 != 0) return PASA_ERR_UNSUPPORTED;
    if (!aligned16(planes[i]) || !aligned16(out_planes[i])) return PASA_ERR_ALIGN;
    in_place |= planes[i] == out_planes[i];
    apart |= planes[i] != out_planes[i];
    // a plane listed twice would be moved by two CTAs at once
    if (out_planes[i] == static_cast<void*>(out_weights)) return PASA_ERR_SHAPE;
    for (int j = 0; j < i; ++j)
      if (out_planes[i] == out_planes[j]) return PASA_ERR_SHAPE;
  }
  // a cache moves in place as a whole, in a cache of the same size
  if (in_place && (apart || out_cap != Sk_cap)) return PASA_ERR_SHAPE;
  // else a row could be written over before it is read, by another CTA. In place a tensor meets itself only.
  const unsigned long long heads = static_cast<unsigned long long>(B) * Hkv;
  Span from[pasa::kEvictPlanes + 1], to[pasa::kEvictPlanes + 1];
  for (int i = 0; i < n_planes; ++i) {
    from[i] = Span(planes[i], heads * Sk_cap, row_bytes[i]);
    to[i] = Span(out_planes[i], heads * out_cap, row_bytes[i]);
  }
  from[n_planes] = Span(weights, heads * Sk_cap, 4);
  to[n_planes] = Span(out_weights, heads * out_cap, 4);
  for (int i = 0; i <= n_planes; ++i)
    for (int j = 0; j <= n_planes; ++j)
      if ((i != j || !in_place) && (to[i].meets(from[j]) || (i < j && to[i].meets(to[j])))) return PASA_ERR_SHAPE;
  pasa::EvictPlanes pl = {};
  pl.n = n_planes + 1;
  long long blocks = 0;
  for (int i = 0; i <= n_planes; ++i) {
    const bool w = i == n_planes;
    pl.src[i] = static_cast<const unsigned char*>(w ? static_cast<const void*>(weights) : planes[i]);
    pl.dst[i] = static_cast<unsigned char*>(w ? static_cast<void*>(out_weights) : out_planes[i]);
    pl.row_bytes[i] = w ? 4 : row_bytes[i];
    pl.width[i] = in_place ? 32 : 128;
    const int rows = pasa::move_rows_per_round(pl.row_bytes[i], pl.width[i]);
    pl.parts[i] = in_place ? 1 : static_cast<int>((static_cast<long long>(budget) + rows - 1) / rows);
    blocks += static_cast<long long>(pl.parts[i]) * ((pl.row_bytes[i] + pl.width[i] - 1) / pl.width[i]);
    if (blocks > 65535) return PASA_ERR_SHAPE;   // grid.y
    pl.first[i + 1] = static_cast<int>(blocks);
  }
  if (Sk > INT_MAX - 65536 || budget > INT_MAX - 65536) return PASA_ERR_SHAPE;   // row numbers of a round
  int rc = check_device();
  if (rc != PASA_OK) return rc;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned planes_bh = static_cast<unsigned>(B) * static_cast<unsigned>(Hkv);
  // CTAs of a head: more while each has over 4096 rows and all fit the SMs one to each
  int cluster = 1;
  while (cluster < pasa::kEvictCluster && Sk > cluster * 4096 && planes_bh * cluster * 2 <= 152) cluster *= 2;
  static std::atomic<unsigned long long> raised{0};
  cudaError_t e = launch_clusters(pasa::evict_select_kernel, planes_bh * cluster, pasa::kEvictThreads, 0, 0, st, false,
                                  cluster, raised, weights, lengths, index, Hkv, Sk, static_cast<long long>(Sk_cap), budget,
                                  recent, cluster);
  if (e != cudaSuccess) return cuda_fail(e);
  const dim3 grid(planes_bh, pl.first[pl.n]);
  e = launch_kernel(pasa::evict_move_kernel, grid, dim3(pasa::kMoveThreads), 0, st, true, pl, index,
                                      new_lengths, Hkv, static_cast<long long>(Sk_cap), static_cast<long long>(out_cap),
                                      budget);
  return e == cudaSuccess ? launch_status() : cuda_fail(e);
}

}  // extern "C"
