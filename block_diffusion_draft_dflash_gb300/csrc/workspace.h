// Carving of a caller's workspace and small argument checks, shared by the C ABI entry points.
#pragma once
#include <stddef.h>
#include <stdint.h>

#include "../../include/dflash.h"

namespace df {
namespace {
constexpr size_t kAlign = 256;
inline size_t up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }

// Bump allocator over a caller-provided workspace (or a size counter when base is null).
struct Carver {
  unsigned char* base;
  size_t off = kAlign;  // the first 256 bytes hold the status header
  explicit Carver(void* b) : base(static_cast<unsigned char*>(b)) {}
  template <class T>
  T* take(size_t count) {
    T* p = base ? reinterpret_cast<T*>(base + off) : nullptr;
    off = up(off + count * sizeof(T));
    return p;
  }
};

inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline int* status_of(void* ws) { return reinterpret_cast<int*>(ws); }

#define DF_TRY(x)            \
  do {                       \
    int _rc = (x);           \
    if (_rc != DF_OK) return _rc; \
  } while (0)
}  // namespace
}  // namespace df
