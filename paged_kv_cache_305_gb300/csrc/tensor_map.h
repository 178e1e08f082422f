// Host side: the driver's tensor-map encoder and kernel attributes, looked up and
// set once.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <atomic>

namespace pa {

// A driver entry as of CUDA 12.0; null if the driver does not have it.
template <typename Fn>
inline Fn driver_entry(const char* name, std::atomic<Fn>& fn) {
  Fn f = fn.load(std::memory_order_acquire);
  if (f == nullptr) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion(name, &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess && p != nullptr) {
      f = reinterpret_cast<Fn>(p);
      fn.store(f, std::memory_order_release);
    }
  }
  return f;
}

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> fn{nullptr};
  return driver_entry("cuTensorMapEncodeTiled", fn);
}

// Sets attributes of a kernel, which belong to a context and stay set in it: calls
// `set` unless `done` names the current context (an id that no later context gets).
template <typename F>
inline cudaError_t once_per_context(std::atomic<unsigned long long>& done, F set) {
  static std::atomic<PFN_cuCtxGetId_v12000> fn{nullptr};
  const PFN_cuCtxGetId_v12000 get_id = driver_entry("cuCtxGetId", fn);
  unsigned long long id = 0;
  const bool known = get_id != nullptr && get_id(nullptr, &id) == CUDA_SUCCESS;
  if (known && done.load(std::memory_order_acquire) == id + 1) return cudaSuccess;
  const cudaError_t e = set();
  if (e == cudaSuccess && known) done.store(id + 1, std::memory_order_release);
  return e;
}

}  // namespace pa
