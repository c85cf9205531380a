// Host-side helpers shared by the library's translation units.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/tl.h"

namespace tl {

// Records the CUDA error text for tl_last_cuda_error() and maps it to a status.
int check_cuda(cudaError_t e);

// A buffer of a call, and whether two of them share a byte (NULL and empty ones share none).
struct Buf {
  const void* p;
  size_t bytes;
};
inline bool share_bytes(const Buf& a, const Buf& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && a.bytes && b.bytes && (x < y ? y - x < a.bytes : x - y < b.bytes);
}

// Whether a tl_kv_pool is one that the serving operators take.
bool kv_pool_ok(const tl_kv_pool* p);

}  // namespace tl

#define TL_CUDA(call)                        \
  do {                                       \
    int _st = ::tl::check_cuda((call));      \
    if (_st != TL_OK) return _st;            \
  } while (0)

#define TL_TRY(call)                         \
  do {                                       \
    int _st = (call);                        \
    if (_st != TL_OK) return _st;            \
  } while (0)
