// Host-side helpers shared by the library's translation units: the thread's error
// text, argument checks, launches of the dependent-launch chains, device queries.
#pragma once

#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <array>
#include <cstdarg>
#include <cstdio>
#include <mutex>
#include <string>
#include <utility>
#include <vector>

#include "dfssm.h"

namespace dfssm {

// Message of the calling thread's last failure (dfssm_last_error).
inline std::string& last_error_text() {
  static thread_local std::string text;
  return text;
}

inline int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
inline int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  last_error_text() = buf;
  return code;
}

inline int ok() {
  last_error_text().clear();
  return DFSSM_OK;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

#define REQUIRE(cond, code, ...) \
  do {                           \
    if (!(cond)) return fail(code, __VA_ARGS__); \
  } while (0)

#define REQUIRE_PTR(p) \
  do { \
    REQUIRE((p) != nullptr, DFSSM_ERR_INVALID_ARG, "%s is NULL", #p); \
    REQUIRE(aligned16(p), DFSSM_ERR_MISALIGNED, "%s is not 16-byte aligned", #p); \
  } while (0)

#define CHECK_LAUNCH(what) \
  do { \
    cudaError_t e_ = cudaGetLastError(); \
    if (e_ != cudaSuccess) return fail(DFSSM_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e_)); \
  } while (0)

// Kernels of the multi-launch chain are launched with programmatic stream
// serialization: each may start while the kernel before it still runs, does its setup
// and reads only weights until pdl_wait() (common.cuh), so the launch and the setup
// overlap the previous kernel's tail.  DFSSM_PDL=0 at compile time turns it off.
#ifndef DFSSM_PDL
#define DFSSM_PDL 1
#endif
template <typename... KArgs, typename... Args>
cudaError_t launch_chain(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                         dim3 cluster /* x = 0: none */, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  unsigned n = 0;
  if (DFSSM_PDL) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  if (cluster.x > 0) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = cluster.x;
    at[n].val.clusterDim.y = cluster.y;
    at[n].val.clusterDim.z = cluster.z;
    ++n;
  }
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}
#define CHAIN_LAUNCH(what, ...) \
  do { \
    cudaError_t e_ = launch_chain(__VA_ARGS__); \
    if (e_ != cudaSuccess) return fail(DFSSM_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e_)); \
  } while (0)

// Workspace layout: regions one behind the other at 256-byte boundaries.
inline size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

struct Bump {
  size_t off = 0;
  size_t take(size_t bytes) {
    off = align256(off);
    size_t at = off;
    off += bytes;
    return at;
  }
};

inline int current_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    dev = 0;
  }
  return dev;
}

// SM count of the current device, cached per device.
inline int sm_count() {
  static std::mutex mu;
  static std::vector<std::array<int, 2>> cache;   // device, SMs
  const int dev = current_device();
  std::lock_guard<std::mutex> lock(mu);
  for (const auto& c : cache)
    if (c[0] == dev) return c[1];
  int v = 0;
  if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0) {
    cudaGetLastError();
    v = 148;
  }
  cache.push_back({dev, v});
  return v;
}

// cuTensorMapEncodeTiled through the runtime's driver entry point (no link against
// the driver library), looked up once.  It wants a current context, which a host thread
// has only after its first call that needs one: setting the thread's device gives it one
// (and, unlike an allocation, may be done while a stream is being captured).
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  thread_local bool bound = false;
  if (!bound) {
    int dev = 0;
    bound = cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess;
  }
  return fn;
}

}  // namespace dfssm
