// cp_call.h -- what the host sides of the calls on caller-owned arrays share:
// the current device kept, checks of addresses and strides, error codes.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <initializer_list>

#include "cp.h"

namespace cp {

struct DeviceGuard {
  int prev = -1;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
    if (prev == dev) prev = -1;
    else cudaSetDevice(dev);
  }
  ~DeviceGuard() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Whether the entries of a strided array, `row` elements each, lie apart: from the smallest stride up, each passes
// all that the ones below it span.
struct Axis {
  int64_t n, stride;
};
inline bool lie_apart(int64_t row, std::initializer_list<Axis> axes) {
  Axis a[3];
  int m = 0;
  for (const Axis& x : axes)
    if (x.n > 1) a[m++] = x;
  std::sort(a, a + m, [](const Axis& x, const Axis& y) { return x.stride < y.stride; });
  for (int i = 0; i < m; ++i) {
    if (a[i].stride < row) return false;
    if (i + 1 < m) {                                   // row + (n - 1) * stride, which may pass 64 bits, within the next stride
      if ((a[i + 1].stride - row) / a[i].stride < a[i].n - 1) return false;
      row += (a[i].n - 1) * a[i].stride;
    }
  }
  return true;
}

inline int cuda_err(cudaError_t e) { return e == cudaSuccess ? CP_OK : CP_ERR_CUDA; }

// A function of the driver's, which makes no context of its own: where a thread's first use of CUDA finds none, that of the
// current device is made the thread's, and the function called again.
template <class F>
CUresult in_context(F call) {
  CUresult r = call();
  int device = 0;
  if (r == CUDA_ERROR_INVALID_CONTEXT && cudaGetDevice(&device) == cudaSuccess && cudaSetDevice(device) == cudaSuccess) r = call();
  return r;
}

// CP_OK on an sm_103 device.
inline int check_device(int device) {
  int ndev = 0, major = 0, minor = 0;
  if (cudaGetDeviceCount(&ndev) != cudaSuccess || device < 0 || device >= ndev) {
    cudaGetLastError();
    return CP_ERR_UNSUPPORTED;
  }
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, device) != cudaSuccess)
    return CP_ERR_CUDA;
  return major == 10 && minor == 3 ? CP_OK : CP_ERR_UNSUPPORTED;
}

// Whether `p` is memory of that device.
inline bool on_device(const void* p, int device) {
  cudaPointerAttributes a{};
  if (cudaPointerGetAttributes(&a, p) == cudaSuccess && a.type == cudaMemoryTypeDevice && a.device == device) return true;
  cudaGetLastError();
  return false;
}

// A launch in clusters of cluster_x by cluster_y blocks, and, with `early`, one that may start before the kernel in
// front of it has ended (it waits for that one where it needs to: pdl_wait).
template <class K, class... A>
cudaError_t launch_as(K kernel, dim3 grid, int cluster_x, int cluster_y, bool early, int threads, size_t smem, cudaStream_t s,
                      const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  if (cluster_x * cluster_y > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = cluster_x;
    attr[cfg.numAttrs].val.clusterDim.y = cluster_y;
    attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  if (early) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  cfg.attrs = attr;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace cp
