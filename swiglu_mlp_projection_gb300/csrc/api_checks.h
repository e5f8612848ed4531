// Argument checks that the C-ABI functions of several files share.
#pragma once

#include <stdint.h>
#include <stdio.h>

#include "internal.h"
#include "swiglu.h"

namespace swg {

struct Span {
  const char* name;
  const void* p;
  size_t bytes;
  unsigned align = 16;   // what the kernels' loads of it need
};

inline int failf(int status, const char* fmt, const char* a, const char* b = "") {
  char text[256];
  snprintf(text, sizeof text, fmt, a, b);
  return api_fail(status, text);
}

// Every non-empty tensor has a pointer, aligned as its loads need.
inline int check_spans(const Span* s, int n) {
  for (int i = 0; i < n; ++i) {
    if (s[i].bytes && !s[i].p)
      return failf(SWIGLU_ERR_INVALID_ARG, "null pointer for a non-empty tensor (%s)", s[i].name);
    if ((uintptr_t)s[i].p & (s[i].align - 1))
      return failf(SWIGLU_ERR_ALIGNMENT, "%s must be %s-byte aligned", s[i].name,
                   s[i].align == 16 ? "16" : s[i].align == 4 ? "4" : "2");
  }
  return SWIGLU_OK;
}

inline bool overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
  const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
  return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

inline int check_apart(const Span& out, const Span* s, int n) {
  for (int i = 0; i < n; ++i)
    if (overlap(out, s[i])) return failf(SWIGLU_ERR_INVALID_ARG, "%s overlaps %s", out.name, s[i].name);
  return SWIGLU_OK;
}

// As check_apart, but `out` may be one of the tensors itself.
inline int check_apart_or_same(const Span& out, const Span* s, int n) {
  for (int i = 0; i < n; ++i)
    if (out.p != s[i].p && overlap(out, s[i]))
      return failf(SWIGLU_ERR_INVALID_ARG, "%s partially overlaps %s", out.name, s[i].name);
  return SWIGLU_OK;
}

inline size_t round256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace swg
