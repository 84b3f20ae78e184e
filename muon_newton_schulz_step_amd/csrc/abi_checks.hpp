// Argument checks shared by the C entry points of the operators around the
// step: statuses with a message, the addresses buffers span, overlaps.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <initializer_list>
#include <string>

#include "muon.h"
#include "plan.hpp"

namespace muon {
namespace abi {

constexpr int64_t kMax = (int64_t)1 << 31;  // sizes are below this

inline muon_status fail(muon_status st, const char *where, const char *what) {
  set_error(std::string(where) + ": " + what);
  return st;
}

inline muon_status done(hipError_t e, const char *where) {
  if (e == hipSuccess) return MUON_OK;
  return fail(MUON_ERR_HIP, where, hipGetErrorString(e));
}

// Runs an entry point's body; an exception (host memory for a message) ends
// as a status.
template <class F>
muon_status guarded(F body) {
  try {
    return body();
  } catch (...) {
    return MUON_ERR_INVALID_ARG;
  }
}

inline bool known_dtype(int32_t t) { return t == MUON_DT_FP32 || t == MUON_DT_BF16; }
inline bool known_index(int32_t t) { return t == MUON_IDX_INT32 || t == MUON_IDX_INT64; }
inline uintptr_t dtype_bytes(int32_t t) { return t == MUON_DT_BF16 ? 2 : 4; }
inline uintptr_t index_bytes(int32_t t) { return t == MUON_IDX_INT64 ? 8 : 4; }

// The addresses a buffer spans.
struct Span {
  uintptr_t lo, hi;
  const char *name;
};
inline Span flat(const void *p, int64_t n, uintptr_t e, const char *name) {
  return {(uintptr_t)p, (uintptr_t)p + (p ? (uintptr_t)n * e : 0), name};
}
inline Span matrix(const void *p, int64_t rows, int64_t cols, int64_t ld, uintptr_t e, const char *name) {
  return flat(p, rows > 0 ? (rows - 1) * ld + cols : 0, e, name);
}

// Whether a rows x ld extent stays an address (2^62 bytes leave room).
inline bool fits(int64_t rows, int64_t ld) { return ld < ((int64_t)1 << 59) && (rows == 0 || ld < ((int64_t)1 << 59) / rows); }

// Every written buffer against every other buffer of the call.
inline muon_status no_overlap(const char *where, std::initializer_list<Span> out, std::initializer_list<Span> in) {
  for (const Span *a = out.begin(); a != out.end(); ++a) {
    auto clash = [&](const Span &b) { return a->lo < a->hi && b.lo < b.hi && a->lo < b.hi && b.lo < a->hi; };
    for (const Span *b = a + 1; b != out.end(); ++b)
      if (clash(*b)) {
        set_error(std::string(where) + ": buffers overlap: " + a->name + " and " + b->name);
        return MUON_ERR_ALIAS;
      }
    for (const Span &b : in)
      if (clash(b)) {
        set_error(std::string(where) + ": buffers overlap: " + a->name + " and " + b.name);
        return MUON_ERR_ALIAS;
      }
  }
  return MUON_OK;
}

inline muon_status check_workspace(const char *where, const void *ws, size_t have, size_t need) {
  if (!ws) return fail(MUON_ERR_WORKSPACE, where, "workspace is NULL");
  if ((uintptr_t)ws % 256 != 0) return fail(MUON_ERR_WORKSPACE, where, "workspace must be 256-byte aligned");
  if (have < need) {
    set_error(std::string(where) + ": workspace too small: " + std::to_string(have) + " < " + std::to_string(need));
    return MUON_ERR_WORKSPACE;
  }
  return MUON_OK;
}

}  // namespace abi
}  // namespace muon
