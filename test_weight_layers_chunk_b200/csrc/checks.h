// Host-side argument checks shared by the C entry points: failure reporting
// through e2ttt_last_error(), alignment, and overlap of outputs with inputs.
#pragma once
#include <cuda_runtime.h>
#include <stdarg.h>
#include <stddef.h>
#include <stdint.h>
#include <stdio.h>

#include <initializer_list>

#include "../../include/e2ttt.h"

namespace e2ttt {

// The calling thread's e2ttt_last_error() text (api.cu).
void set_last_error(const char* msg);

inline e2ttt_status failf(e2ttt_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
inline e2ttt_status failf(e2ttt_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  set_last_error(buf);
  return s;
}

inline e2ttt_status fail_cuda(cudaError_t e, const char* where) {
  return failf(E2TTT_ERR_CUDA, "%s: %s (%s)", where, cudaGetErrorName(e), cudaGetErrorString(e));
}

struct Span {
  const void* p;
  size_t n;  // bytes
  const char* name;
};

inline bool spans_meet(const Span& a, const Span& b) {
  if (!a.p || !b.p || !a.n || !b.n) return false;
  const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
  return a0 < b0 + b.n && b0 < a0 + a.n;
}

// Every output must be disjoint from every input and every other output.
inline e2ttt_status check_spans(const char* who, std::initializer_list<Span> in,
                                std::initializer_list<Span> out) {
  for (const Span* o = out.begin(); o != out.end(); ++o) {
    for (const Span& i : in)
      if (spans_meet(*o, i))
        return failf(E2TTT_ERR_INVALID_ARG, "%s: %s overlaps input %s", who, o->name, i.name);
    for (const Span* p = o + 1; p != out.end(); ++p)
      if (spans_meet(*o, *p))
        return failf(E2TTT_ERR_INVALID_ARG, "%s: %s overlaps output %s", who, o->name, p->name);
  }
  return E2TTT_OK;
}

// Pointers must be aligned to the element they point to: `align` bytes.
inline e2ttt_status check_aligned(const char* who, size_t align, std::initializer_list<Span> ps) {
  for (const Span& s : ps)
    if (((uintptr_t)s.p) & (align - 1))
      return failf(E2TTT_ERR_INVALID_ARG, "%s: %s must be aligned to %zu bytes", who, s.name, align);
  return E2TTT_OK;
}

inline bool all_aligned(size_t align, std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (((uintptr_t)p) & (align - 1)) return false;
  return true;
}

}  // namespace e2ttt
