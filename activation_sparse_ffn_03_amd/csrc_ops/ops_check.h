// Checks of arguments and errors shared by the C ABI files of the operators
// around the block. Host code.
#pragma once

#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include <hip/hip_runtime.h>

#include "../csrc/twell_host.h"
#include "../csrc/twell_internal.h"

namespace twell::check {

inline twell_status fail(twell_status st, const char* why) { return twell::set_error(st, why); }

inline twell_status hip_status(hipError_t e, const char* where) {
  if (e == hipSuccess) return TWELL_OK;
  char why[256];  // no allocation, nothing to throw
  std::snprintf(why, sizeof why, "%s: %s", where, hipGetErrorString(e));
  return twell::set_error(TWELL_ERR_HIP, why);
}

inline twell_status ok() {
  twell::set_error(TWELL_OK, "");
  return TWELL_OK;
}

inline bool bad_dtype(twell_dtype t) { return t != TWELL_BF16 && t != TWELL_F32; }
inline size_t size_of(twell_dtype t) { return t == TWELL_BF16 ? 2 : 4; }

#define OPS_CHECK_PTR(p, bytes, name)                                                            \
  do {                                                                                           \
    if (twell::bad_ptr((p), (bytes)))                                                            \
      return fail(TWELL_ERR_INVALID_ARG, name " is NULL or not 16-byte aligned");                \
  } while (0)
#define OPS_CHECK_OPT(p, bytes, name)                                                            \
  do {                                                                                           \
    if ((p) != nullptr) OPS_CHECK_PTR(p, bytes, name);                                           \
  } while (0)

inline twell_status check_ws(void* ws, size_t have, size_t need, const char* small) {
  if (have < need) return fail(TWELL_ERR_WORKSPACE, small);
  if (twell::bad_ptr(ws, need)) return fail(TWELL_ERR_WORKSPACE, "workspace is NULL or not 16-byte aligned");
  return TWELL_OK;
}

// Memory of an array that a call reads or writes; null: none.
struct Span {
  const void* p;
  size_t bytes;
};
inline bool meet(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x != 0 && y != 0 && a.bytes > 0 && b.bytes > 0 && x < y + b.bytes && y < x + a.bytes;
}
// Refuses outputs that share memory with an input or with each other.
inline twell_status check_apart(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    for (const Span& in : ins)
      if (meet(*o, in)) return fail(TWELL_ERR_INVALID_ARG, "an output overlaps an input");
    for (const Span* p = o + 1; p != outs.end(); ++p)
      if (meet(*o, *p)) return fail(TWELL_ERR_INVALID_ARG, "outputs overlap each other");
  }
  return TWELL_OK;
}

}  // namespace twell::check
