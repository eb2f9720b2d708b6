// Host-side launch helpers shared by the kernel launchers of libpa.so.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>
#include <unordered_map>

namespace pa {

// cuTensorMapEncodeTiled, through the runtime's entry-point query (the library
// does not link the driver); null when there is none.
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// Encodes a tensor map (the arguments are cuTensorMapEncodeTiled's). The driver wants a current
// context, and a thread that has made no runtime call yet has none: cudaSetDevice binds its device's.
template <class... Args>
inline bool encode_tensor_map(Args... args) {
  const auto encode = tensor_map_encoder();
  if (!encode) return false;
  CUresult r = encode(args...);
  int device = 0;
  if (r == CUDA_ERROR_INVALID_CONTEXT && cudaGetDevice(&device) == cudaSuccess &&
      cudaSetDevice(device) == cudaSuccess)
    r = encode(args...);
  return r == CUDA_SUCCESS;
}

// Raise a kernel's dynamic shared-memory limit once per (kernel, device) rather
// than on every launch.
inline cudaError_t ensure_smem_attr(const void* kern, int bytes) {
  static std::mutex mu;
  static std::unordered_map<uint64_t, int> done;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) dev = 0;
  const uint64_t key = (reinterpret_cast<uint64_t>(kern) << 8) ^ uint64_t(dev);
  {
    std::lock_guard<std::mutex> lock(mu);
    auto it = done.find(key);
    if (it != done.end() && it->second >= bytes) return cudaSuccess;
  }
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) {
    std::lock_guard<std::mutex> lock(mu);
    int& v = done[key];
    if (v < bytes) v = bytes;
  }
  return e;
}

}  // namespace pa
