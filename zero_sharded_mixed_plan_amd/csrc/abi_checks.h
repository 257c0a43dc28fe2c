// Argument checks shared by the C ABI of the model's layers (input_abi.cpp,
// layer_abi.cpp).  Included inside a source only.
#pragma once

#include <cstdint>
#include <exception>
#include <new>
#include <string>

#include "zero_internal.h"

namespace {

using zk::fail;

constexpr int64_t kMax31 = int64_t(1) << 31;
constexpr int64_t kMaxLd = int64_t(1) << 40;  // elements; keeps every byte offset within 64 bits

int bytes_of(zero_dtype_t t) {
  switch (t) {
    case ZERO_F32: return 4;
    case ZERO_BF16:
    case ZERO_F16: return 2;
  }
  return 0;
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

struct Span {
  uintptr_t lo, hi;
};

Span span(const void* p, int64_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Span{a, a + (uintptr_t)(p ? bytes : 0)};
}
// a [rows, cols] matrix with rows ld elements apart
Span span(const void* p, int64_t rows, int64_t cols, int64_t ld, int eb) {
  return span(p, rows > 0 ? ((rows - 1) * ld + cols) * eb : 0);
}
const char* end_of(const Span& s) { return reinterpret_cast<const char*>(s.hi); }
bool overlap(const Span& x, const Span& y) { return x.lo < y.hi && y.lo < x.hi; }

// No exception leaves a C entry.
template <class F>
int guarded(F&& f) noexcept {
  try {
    return f();
  } catch (const std::bad_alloc&) {
    return ZERO_ENOMEM;  // no memory for a message either
  } catch (...) {
    return ZERO_EINVAL;
  }
}

int matrix(const char* fn, const char* what, const void* p, int64_t rows, int64_t cols, int64_t ld,
           zero_dtype_t t) {
  const int eb = bytes_of(t);
  if (eb == 0) return fail(ZERO_EINVAL, std::string(fn) + ": unsupported dtype of " + what);
  if (rows == 0) return ZERO_OK;
  if (!p) return fail(ZERO_EINVAL, std::string(fn) + ": " + what + " is NULL");
  if (ld < cols && rows > 1) return fail(ZERO_EINVAL, std::string(fn) + ": the rows of " + what + " overlap (stride < columns)");
  if (ld < 0 || ld > kMaxLd || rows > kMaxLd || (rows > 1 && ld > (int64_t(1) << 60) / rows))
    return fail(ZERO_EINVAL, std::string(fn) + ": the stride of " + what + " is out of range");
  if (!aligned(p, eb)) return fail(ZERO_EALIGN, std::string(fn) + ": " + what + " is not element aligned");
  return ZERO_OK;
}

}  // namespace
