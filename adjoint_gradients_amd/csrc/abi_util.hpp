// abi_util.hpp -- argument checks and the workspace carver shared by the C
// entries of the operators (host side).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/ssm_adjoint.h"

namespace abi {

constexpr size_t kAlign = 256;

inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Required and optional device pointers.
inline bool good(const void* p) { return p && aligned16(p); }
inline bool good_or_null(const void* p) { return aligned16(p); }

// Sequential carve-out of a workspace; with a null base only sizes are summed.
struct Carver {
  char* base;
  size_t off = 0;
  explicit Carver(void* b) : base(static_cast<char*>(b)) {}
  template <typename T> T* take(size_t count) {
    T* p = base ? reinterpret_cast<T*>(base + off) : nullptr;
    off += align_up(count * sizeof(T));
    return p;
  }
};

inline ssm_status check_ws(void* ws, size_t have, size_t need) {
  if (need == 0) return SSM_OK;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & (kAlign - 1)) != 0 || have < need) return SSM_ERR_WORKSPACE;
  return SSM_OK;
}

}  // namespace abi
