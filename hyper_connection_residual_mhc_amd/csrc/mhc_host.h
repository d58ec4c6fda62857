// mhc_host.h - host-side argument checks shared by the norm, product and
// write-back libraries (internal; not part of the C ABI): the thread's error
// text, pointer and overlap tests, and launch status.

#pragma once

#include <hip/hip_runtime.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "mhc_h_aggregate.h"

namespace {

thread_local char g_msg[256] = "";

mhc_status fail(mhc_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
mhc_status fail(mhc_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
  va_end(ap);
  return s;
}

mhc_status ok() {
  g_msg[0] = '\0';
  return MHC_SUCCESS;
}

// One tensor argument of a call. `bytes` < 0 marks a size that does not fit
// 64 bits; an absent optional tensor has a null pointer and 0 bytes.
struct Tensor {
  const void* p;
  int64_t bytes;
  int64_t align;
  const char* name;
};

// a * b * c for non-negative factors, or -1 past int64.
int64_t mul_bytes(int64_t a, int64_t b, int64_t c) {
  int64_t r;
  if (a < 0 || b < 0 || c < 0 || __builtin_mul_overflow(a, b, &r) ||
      __builtin_mul_overflow(r, c, &r))
    return -1;
  return r;
}

mhc_status check_tensor(const Tensor& t) {
  if (t.bytes < 0)
    return fail(MHC_ERROR_INVALID_VALUE, "the size of %s does not fit 64 bits", t.name);
  if (t.bytes > 0 && t.p == nullptr) return fail(MHC_ERROR_INVALID_VALUE, "%s is NULL", t.name);
  if (reinterpret_cast<uintptr_t>(t.p) % static_cast<uintptr_t>(t.align) != 0)
    return fail(MHC_ERROR_INVALID_VALUE, "%s is not %lld-byte aligned", t.name,
                static_cast<long long>(t.align));
  if (reinterpret_cast<uintptr_t>(t.p) + static_cast<uintptr_t>(t.bytes) <
      reinterpret_cast<uintptr_t>(t.p))
    return fail(MHC_ERROR_INVALID_VALUE, "%s runs past the address space", t.name);
  return ok();
}

bool overlap(const Tensor& a, const Tensor& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + static_cast<uintptr_t>(b.bytes) && y < x + static_cast<uintptr_t>(a.bytes);
}

// Every tensor is present and aligned, and no output overlaps an input or
// another output.
template <int I, int O>
mhc_status check_tensors(const Tensor (&in)[I], const Tensor (&out)[O]) {
  mhc_status st;
  for (const Tensor& t : in)
    if ((st = check_tensor(t)) != MHC_SUCCESS) return st;
  for (const Tensor& t : out)
    if ((st = check_tensor(t)) != MHC_SUCCESS) return st;
  for (int a = 0; a < O; ++a) {
    for (int b = 0; b < I; ++b)
      if (overlap(out[a], in[b]))
        return fail(MHC_ERROR_ALIASING, "output %s overlaps input %s", out[a].name, in[b].name);
    for (int b = a + 1; b < O; ++b)
      if (overlap(out[a], out[b]))
        return fail(MHC_ERROR_ALIASING, "output %s overlaps output %s", out[a].name, out[b].name);
  }
  return ok();
}

// The status of one launch or event call (the value it returned itself).
mhc_status launch_status(hipError_t e, const char* what) {
  if (e != hipSuccess)
    return fail(MHC_ERROR_HIP, "%s failed: %s (%s)", what, hipGetErrorName(e),
                hipGetErrorString(e));
  return ok();
}

// A call with no work: both events, where given, with nothing between them.
mhc_status record_empty(void* stream, void* start, void* stop) {
  hipError_t e = hipSuccess;
  if (start != nullptr)
    e = hipEventRecord(static_cast<hipEvent_t>(start), static_cast<hipStream_t>(stream));
  if (e == hipSuccess && stop != nullptr)
    e = hipEventRecord(static_cast<hipEvent_t>(stop), static_cast<hipStream_t>(stream));
  return launch_status(e, "event record");
}

}  // namespace
