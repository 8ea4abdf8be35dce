// Argument checks shared by the C ABI's source files around the layer.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstddef>
#include <cstdint>
#include <cstdio>

#include "api_internal.h"

namespace moe {
namespace api {

inline moe_status_t fail(moe_status_t s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return moe::set_error(s, buf);
}

inline moe_status_t done(hipError_t e, const char* where) {
  if (e != hipSuccess) return fail(MOE_ERR_HIP, "%s: %s", where, hipGetErrorString(e));
  return moe::set_error(MOE_OK, "");
}

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

constexpr size_t kAlign = 256;
inline size_t up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

inline moe_status_t check_workspace(const void* ws, size_t have, size_t need) {
  if (!ws || !aligned(ws, kAlign))
    return fail(MOE_ERR_INVALID_ARGUMENT, "workspace must be non-NULL and 256-byte aligned");
  if (have < need)
    return fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace %zu < required %zu", have, need);
  return MOE_OK;
}

inline moe_status_t check_aligned(const void* const* p, int count, size_t a, const char* what) {
  for (int i = 0; i < count; ++i)
    if (p[i] && !aligned(p[i], a))
      return fail(MOE_ERR_INVALID_ARGUMENT, "%s must be %zu-byte aligned", what, a);
  return MOE_OK;
}

// A buffer of a call (p NULL: absent).  inplace: the input and the output that
// may be one buffer.
struct Span {
  const void* p;
  size_t bytes;
  bool inplace = false;
};

// No output (the workspace is one) shares memory with an input or another
// output: a launch would overwrite what a later one still reads.
inline moe_status_t check_alias(const Span* in, int n_in, const Span* out, int n_out) {
  auto share = [](const Span& a, const Span& b) {
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return a.p && b.p && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
  };
  for (int o = 0; o < n_out; ++o) {
    for (int i = 0; i < n_in; ++i)
      if (share(in[i], out[o]) && !(in[i].inplace && out[o].inplace && in[i].p == out[o].p))
        return fail(MOE_ERR_INVALID_ARGUMENT, "an output aliases an input");
    for (int j = 0; j < o; ++j)
      if (share(out[j], out[o]))
        return fail(MOE_ERR_INVALID_ARGUMENT, "two outputs alias each other");
  }
  return MOE_OK;
}

template <int I, int O>
moe_status_t check_alias(const Span (&in)[I], const Span (&out)[O]) {
  return check_alias(in, I, out, O);
}

}  // namespace api
}  // namespace moe
