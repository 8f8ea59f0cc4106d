// pi_host.cuh -- host-side helpers shared by the C ABI's source files.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>

#include "pi_ffn.h"

#define PI_CUDA(call)                                   \
  do {                                                 \
    if ((call) != cudaSuccess) return PI_ERR_CUDA;     \
  } while (0)

namespace pi {
namespace host {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// A once-per-device setup step (a kernel's function attribute acts on the
// current device only): one bit per device ordinal below 64.
class DeviceOnce {
 public:
  // runs set() unless it already succeeded on the current device
  template <typename Set>
  cudaError_t ensure(Set set) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    const unsigned long long bit = 1ull << dev;
    if (bits_.load(std::memory_order_acquire) & bit) return cudaSuccess;
    if ((e = set()) != cudaSuccess) return e;
    bits_.fetch_or(bit, std::memory_order_acq_rel);
    return cudaSuccess;
  }

 private:
  std::atomic<unsigned long long> bits_{0};
};

inline int device_sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

// Test support (pi_debug_wait_fault): an entry of h that is never published (or,
// for the dense products, finished accumulators that are never announced),
// and a shorter limit for every bounded wait of the fused, batch and dense
// kernels.
struct WaitFault {
  int withhold = -1;
  unsigned long long limit_ns = 0;  // 0: the kernel's default
};
inline WaitFault g_wait_fault;

// cuTensorMapEncodeTiled through the runtime's driver entry point (no link
// against the driver library); null when no driver is present.
using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeTiledFn encoder() {
  static EncodeTiledFn fn = []() -> EncodeTiledFn {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || !p) {
      cudaGetLastError();
      return nullptr;
    }
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

// 2D map of a row-major matrix [rows x inner] of 1- or 2-byte elements, box
// [box_rows x box_inner]; 128-byte swizzle when swz.  Outside reads are zero.
inline bool map_2d(CUtensorMap *m, const void *base, bool fp16, uint64_t inner, uint64_t rows, uint32_t box_inner,
            uint32_t box_rows, bool swz) {
  EncodeTiledFn enc = encoder();
  if (!enc) return false;
  const uint64_t esz = fp16 ? 2 : 1;
  const cuuint64_t dims[2] = {inner, rows};
  const cuuint64_t strides[1] = {inner * esz};
  const cuuint32_t box[2] = {box_inner, box_rows};
  const cuuint32_t es[2] = {1, 1};
  auto encode = [&] {
    return enc(m, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base),
               dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               swz ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = encode();
  if (r == CUDA_ERROR_INVALID_CONTEXT) {
    // A driver call, which finds no context in a host thread that has made no
    // runtime call of the kind that takes the device's: take it, and again.
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess) return false;
    r = encode();
  }
  return r == CUDA_SUCCESS;
}

// ---------------------------------------------------------------- dense block operators
constexpr size_t kHeader = 256;      // start of a workspace: its status word
constexpr int kMaxTokens = 1 << 24;  // tile and row indices stay in 32 bits

inline int cdiv(int a, int b) { return (a + b - 1) / b; }
inline bool overlap(const void *p, size_t pn, const void *q, size_t qn) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p && q && pn && qn && a < b + qn && b < a + pn;
}
// Memory of an argument (null: none).
struct Range {
  const void *p;
  size_t n;
};
// whether one of the first n_out ranges (outputs) shares memory with another of the n
inline bool overlapping(const Range *r, int n_out, int n) {
  for (int i = 0; i < n_out; ++i)
    for (int j = i + 1; j < n; ++j)
      if (overlap(r[i].p, r[i].n, r[j].p, r[j].n)) return true;
  return false;
}
inline bool is_half(int t) { return t == PI_DT_F16 || t == PI_DT_BF16; }
inline bool is_type(int t) { return t == PI_DT_F32 || is_half(t); }
inline size_t type_size(int t) { return t == PI_DT_F32 ? 4 : 2; }

// Launches a kernel with one argument as a programmatic dependent of the
// work before it (the kernel waits by griddepcontrol.wait).  cluster: cluster
// size, 0 for the kernel's own; once: set where the kernel uses dynamic shared
// memory, up to max_smem.
template <typename KArg>
cudaError_t launch1(void (*kern)(KArg), dim3 grid, int threads, size_t smem, int cluster, DeviceOnce *once,
                    cudaStream_t st, const KArg &arg, int max_smem = 224 * 1024) {
  if (once) {
    const cudaError_t e = once->ensure(
        [&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, max_smem); });
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, arg);
}

}  // namespace host
}  // namespace pi
