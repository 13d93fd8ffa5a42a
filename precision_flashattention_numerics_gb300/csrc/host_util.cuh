// Host-side pieces that the library's translation units share: error codes, argument checks, memory
// spans, TMA descriptors, launches.
#pragma once

#include <atomic>
#include <climits>
#include <cstddef>
#include <cstdint>
#include <cstring>
#include <initializer_list>
#include <utility>
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include "../../include/pasa.h"
#include "ptx.cuh"

namespace pasa {

extern thread_local int t_last_cuda_error;   // pasa_last_cuda_error

// The units with bounded waits besides pasa_lib.cu: take_device_error and launch_wait_selftest (below) of each one's
// own device error record, for pasa_check_device_error and pasa_selftest_wait_timeout.
int packed_take_device_error(DeviceError* found);
int packed_wait_selftest(cudaStream_t st);
int tree_take_device_error(DeviceError* found);
int tree_wait_selftest(cudaStream_t st);

}  // namespace pasa

namespace {

using pasa::t_last_cuda_error;

int cuda_fail(cudaError_t e) {
  t_last_cuda_error = static_cast<int>(e);
  return PASA_ERR_CUDA;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

// 3-D fp16 view [planes, rows, D] of a contiguous tensor, 128-byte swizzled boxes of
// 64 x box_rows x 1 elements.
// 3-D map (D, rows, planes) with 128-byte rows per box chunk: 64 fp16 or 128 one-byte elements.
// 3-D map over [planes][rows][D] with planes stride_rows rows apart (0: rows, dense).
int make_map(CUtensorMap* m, const void* base, int D, long long rows, long long planes, int box_rows,
             int elem_bytes = 2, long long stride_rows = 0) {
  auto enc = encode_fn();
  if (!enc) return cuda_fail(cudaErrorNotSupported);
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(planes)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * elem_bytes, static_cast<cuuint64_t>(stride_rows > 0 ? stride_rows : rows) * D * elem_bytes};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / elem_bytes), static_cast<cuuint32_t>(box_rows), 1};
  cuuint32_t es[3] = {1, 1, 1};
  CUresult r = enc(m, elem_bytes == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                   const_cast<void*>(base), dims, strides, box, es,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return cuda_fail(cudaErrorInvalidValue);
  return PASA_OK;
}

int check_device() {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  return pasa_device_supported(dev) ? PASA_OK : PASA_ERR_UNSUPPORTED;
}

// Launch `kern` on `st`; with pdl, by programmatic stream serialization: the kernel may start
// while the kernel queued just ahead of it (the key preparation of the same call) still
// runs, and waits for it with griddep_wait() before reading what it writes.
template <typename... Params, typename... Args>
cudaError_t launch_kernel(void (*kern)(Params...), dim3 grid, dim3 block, int smem, cudaStream_t st, bool pdl,
                          Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  if (pdl) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The memory of a tensor: rows * row_bytes bytes from `at` on (to the last address, if that is past it); none
// for a null pointer. Two spans meet where they share a byte.
struct Span {
  uintptr_t begin = 0, end = 0;
  Span() = default;
  Span(const void* at, unsigned long long rows, unsigned long long row_bytes) {
    if (!at) return;
    unsigned long long bytes;
    begin = reinterpret_cast<uintptr_t>(at);
    if (__builtin_mul_overflow(rows, row_bytes, &bytes) || __builtin_add_overflow(begin, bytes, &end)) end = UINTPTR_MAX;
  }
  bool meets(const Span& x) const { return begin < x.end && x.begin < end; }
};

// Whether `out` shares memory with one of `others`, or two of its own do.
bool any_meet(std::initializer_list<Span> out, std::initializer_list<Span> others) {
  for (const Span* a = out.begin(); a != out.end(); ++a) {
    for (const Span* b = a + 1; b != out.end(); ++b)
      if (a->meets(*b)) return true;
    for (const Span& b : others)
      if (a->meets(b)) return true;
  }
  return false;
}

int launch_status() {
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? PASA_OK : cuda_fail(e);
}

// Launch `kern` in clusters of `cluster` CTAs with `smem` bytes of dynamic shared memory, `max_smem`
// at most in any call. The limit on those is raised at the first launch on a device (bit of
// `raised`), and again if a launch fails (the device was reset).
template <typename... Params>
cudaError_t launch_clusters(void (*kern)(Params...), unsigned grid, int block, int smem, int max_smem,
                            cudaStream_t st, bool pdl, int cluster, std::atomic<unsigned long long>& raised, Params... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  if (pdl) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = cluster;
    attr[cfg.numAttrs].val.clusterDim.y = 1;
    attr[cfg.numAttrs++].val.clusterDim.z = 1;
  }
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (dev < 64 && (raised.load(std::memory_order_relaxed) & bit) != 0) {
    e = cudaLaunchKernelEx(&cfg, kern, args...);
    if (e == cudaSuccess) return e;
    (void)cudaGetLastError();
  }
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, max_smem);
  if (e != cudaSuccess) return e;
  e = cudaLaunchKernelEx(&cfg, kern, args...);
  if (e == cudaSuccess) raised.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// The cache tensors and sizes that every kv4 entry point takes.
int kv4_validate(const void* k4, const void* kscale, const void* v4, const void* vscale, const void* shift, int B,
                 int Hkv, int Sk_cap, int D) {
  if (!k4 || !kscale || !v4 || !vscale) return PASA_ERR_NULLPTR;
  if (B <= 0 || Hkv <= 0 || Sk_cap <= 0) return PASA_ERR_SHAPE;
  if (static_cast<long long>(B) * Hkv > INT_MAX) return PASA_ERR_SHAPE;
  if (D != 64 && D != 128) return PASA_ERR_UNSUPPORTED;
  if (!aligned16(k4) || !aligned16(kscale) || !aligned16(v4) || !aligned16(vscale) || !aligned16(shift))
    return PASA_ERR_ALIGN;
  return PASA_OK;
}

// A call's cache tensors.
struct Kv4Spans {
  Span k4, kscale, v4, vscale, shift;
  Kv4Spans(const void* k4p, const void* ksp, const void* v4p, const void* vsp, const void* shiftp, int B, int Hkv, int cap, int D) {
    const unsigned long long heads = static_cast<unsigned long long>(B) * Hkv, rows = heads * cap;
    k4 = Span(k4p, rows, D / 2), v4 = Span(v4p, rows, D / 2);
    kscale = Span(ksp, rows, D / 16), vscale = Span(vsp, rows, D / 16);
    shift = Span(shiftp, heads, 2 * D);
  }
};

// A strided tensor [B, H, S, D] in bytes, for questions of shared memory.
struct Strided {
  uintptr_t at;
  long long stride[3], n[3];   // of the dimensions, largest stride first
  long long given[6];          // strides and sizes of b, h and s
  long long row;               // bytes of a row

  Strided(const void* p, const long long* strides, long long B, long long H, long long S, long long D, long long size)
      : at(reinterpret_cast<uintptr_t>(p)), stride{strides[0] * size, strides[1] * size, strides[2] * size}, n{B, H, S}, row(D * size) {
    for (int i = 0; i < 3; ++i)
      if (n[i] == 1) stride[i] = 0;   // a dimension of one has no stride
    for (int i = 0; i < 3; ++i) given[i] = stride[i], given[3 + i] = n[i];
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
  // Whether every element of the one is the other's of the same place: the sorted strides do not tell, as a transposed view
  // with two equal sizes has the same ones.
  bool same(const Strided& x) const { return at == x.at && row == x.row && std::memcmp(given, x.given, sizeof given) == 0; }
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

// A map of a strided fp16 tensor: its dimensions, channels first, the strides of the others in bytes, and the box;
// 128-byte swizzle, elements past the tensor read as zeros.
int make_strided_map(CUtensorMap* m, const void* base, std::initializer_list<long long> dims,
                     std::initializer_list<long long> strides, std::initializer_list<long long> box) {
  auto enc = encode_fn();
  if (!enc) return cuda_fail(cudaErrorNotSupported);
  cuuint64_t d[5], st[4];
  cuuint32_t bx[5], es[5] = {1, 1, 1, 1, 1};
  int n = 0;
  for (long long x : dims) d[n++] = static_cast<cuuint64_t>(x);
  int i = 0;
  for (long long x : strides) st[i++] = static_cast<cuuint64_t>(x);
  i = 0;
  for (long long x : box) bx[i++] = static_cast<cuuint32_t>(x);
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, static_cast<cuuint32_t>(n), const_cast<void*>(base), d, st, bx, es,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PASA_OK : cuda_fail(cudaErrorInvalidValue);
}

// Ask for an SM's memory to be split for `kern` as for the kernels with all of its shared memory that run next to it on the
// stream: an SM whose split changes runs empty first. Once per device (bit of `asked`).
template <typename... Params>
void prefer_shared(void (*kern)(Params...), std::atomic<unsigned long long>& asked) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return;
  const unsigned long long bit = 1ull << dev;
  if ((asked.load(std::memory_order_relaxed) & bit) != 0) return;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) == cudaSuccess)
    asked.fetch_or(bit, std::memory_order_relaxed);
}

// This unit's error record, read and cleared: PASA_OK, PASA_ERR_TIMEOUT or PASA_ERR_CUDA.
int take_device_error(pasa::DeviceError* found) {
  cudaError_t e = cudaMemcpyFromSymbol(found, pasa::g_device_error, sizeof *found);
  if (e != cudaSuccess) return cuda_fail(e);
  if (found->word == pasa::kDeviceOk) return PASA_OK;
  const pasa::DeviceError none = {};
  e = cudaMemcpyToSymbol(pasa::g_device_error, &none, sizeof none);
  return e == cudaSuccess ? PASA_ERR_TIMEOUT : cuda_fail(e);
}

// The failure-detection path without a fault: thread 0 waits, through the bounded mbarrier
// wait every kernel of this library uses, on a barrier that nothing arrives on. The wait
// gives up after kWaitTimeoutNs, records the timeout in this unit's record and returns;
// the CTA holds no TMA copy and no tensor memory, so it simply ends. Units' launches behind one another overlap.
__global__ void wait_selftest_kernel() {
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  pasa::griddep_launch_dependents();
  if (threadIdx.x == 0) {
    abort_flag = 0;
    pasa::mbar_init(&bar, 1);
    pasa::fence_mbar_init();
    (void)pasa::mbar_wait(&bar, 0, &abort_flag, 0x5E1F7E57u);   // the self-test's site tag
  }
  pasa::griddep_wait();
}
int launch_wait_selftest(cudaStream_t st, bool pdl) {
  const cudaError_t e = launch_kernel(wait_selftest_kernel, dim3(1), dim3(32), 0, st, pdl);
  return e == cudaSuccess ? launch_status() : cuda_fail(e);
}

}  // namespace
