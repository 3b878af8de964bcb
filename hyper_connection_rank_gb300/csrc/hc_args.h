// Checks of arguments that the C entry points share: every error is found on the
// host, before any launch, and returned as a status.
#pragma once

#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "hc_internal.h"

#define HC_RETURN_IF(expr)                \
  do {                                    \
    const hc_status_t st_ = (expr);       \
    if (st_ != HC_OK) return st_;         \
  } while (0)

namespace hc {
namespace args {

inline hc_status_t fail(hc_status_t s, const char* fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return set_error(s, msg);
}

inline hc_status_t launched(cudaError_t e) {
  return e == cudaSuccess ? HC_OK : fail(HC_ERR_CUDA, "launch: %s", cudaGetErrorString(e));
}

inline bool dtype_valid(int dt) { return dt == HC_F32 || dt == HC_F16 || dt == HC_BF16; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline long long ll(int64_t x) { return static_cast<long long>(x); }

struct Span {
  const char* name;
  uintptr_t lo, hi;
};
inline Span span(const char* name, const void* p, int64_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Span{name, a, p == nullptr || bytes <= 0 ? a : a + static_cast<uintptr_t>(bytes)};
}
inline bool overlaps(const Span& a, const Span& b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }

// No output may overlap an input or another output.
inline hc_status_t check_apart(const Span* outs, int n_out, const Span* ins, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (overlaps(outs[i], ins[j])) return fail(HC_ERR_INVALID_ARG, "%s overlaps %s", outs[i].name, ins[j].name);
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i], outs[j])) return fail(HC_ERR_INVALID_ARG, "%s overlaps %s", outs[i].name, outs[j].name);
  }
  return HC_OK;
}

constexpr int64_t kMaxElems = int64_t{1} << 46;
inline bool sane(int64_t v) { return v >= 0 && v <= kMaxElems; }
// Whether the last of n entries lies within 2^46 elements of the first, so that no sum or product of extents passes 64 bits.
inline bool within(int64_t n, int64_t stride) { return sane(stride) && (n <= 1 || stride <= kMaxElems / (n - 1)); }

// Pointers to tensors lie at a multiple of their element's size.
inline bool on_elements(int dtype, std::initializer_list<const void*> pointers) {
  for (const void* p : pointers)
    if (reinterpret_cast<uintptr_t>(p) % dtype_size(static_cast<hc_dtype_t>(dtype)) != 0) return false;
  return true;
}

// Pointers to 32-bit values.
inline bool on_words(std::initializer_list<const void*> pointers) {
  for (const void* p : pointers)
    if ((reinterpret_cast<uintptr_t>(p) & 3u) != 0) return false;
  return true;
}

inline bool vec_strides(int dtype, std::initializer_list<int64_t> strides) {
  const int64_t v = 16 / static_cast<int64_t>(dtype_size(static_cast<hc_dtype_t>(dtype)));
  for (const int64_t s : strides)
    if (s % v != 0) return false;
  return true;
}

}  // namespace args
}  // namespace hc
