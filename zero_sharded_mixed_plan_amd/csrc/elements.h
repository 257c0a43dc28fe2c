// Element access shared by the kernels that stream matrices (input.hip, norm.hip,
// gated.hip): raw vectors of a type at element-aligned addresses, their values in
// fp32, and results rounded once.  Included inside a kernel source only.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>
#include <type_traits>

#include "input.h"

namespace zk {
namespace {

using u32 = uint32_t;
using u64 = uint64_t;

struct F32 { static constexpr int bytes = 4; };
struct BF16 { static constexpr int bytes = 2; };
struct F16 { static constexpr int bytes = 2; };

typedef u32 vec4 __attribute__((ext_vector_type(4)));
typedef u32 vec2 __attribute__((ext_vector_type(2)));
typedef vec4 vec4_any __attribute__((aligned(2)));  // at an element-aligned address
typedef vec2 vec2_any __attribute__((aligned(2)));

// W consecutive elements, raw
template <class T, int W>
struct Raw {
  u32 w[W * T::bytes / 4];
};

// Loads W elements at p, or, where they would pass `end`, the end of the tensor,
// the W before `end`.  A row's last group reads on into what follows the row, at
// the cost of no further instruction; only the last row's begins early, by the returned
// number of elements, and move_down() puts it right.  The tensor has at least W
// elements (the launches see to it).
template <class T, int W>
__device__ __forceinline__ u32 load_w(const char* p, const char* end, Raw<T, W>& r) {
  constexpr int N = W * T::bytes / 4;
  static_assert(N == 2 || N == 4, "8 or 16 bytes");
  const int64_t past = p + W * T::bytes - end;
  const u32 d = past > 0 ? (u32)past / T::bytes : 0;
  p -= d * T::bytes;
  if constexpr (N == 2) {
    const vec2 q = *reinterpret_cast<const vec2_any*>(p);
    r.w[0] = q.x;
    r.w[1] = q.y;
  } else {
    const vec4 q = *reinterpret_cast<const vec4_any*>(p);
#pragma unroll
    for (int j = 0; j < 4; ++j) r.w[j] = q[j];
  }
  return d;
}

// Moves the elements down by the bits K, K / 2 .. 1 of d; behind the moved ones anything.
template <class T, int W, int K>
__device__ __forceinline__ void move_bits(Raw<T, W>& r, u32 d) {
  constexpr int N = W * T::bytes / 4, M = K * T::bytes / 4;
  const bool on = d & K;
  const Raw<T, W> old = r;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const u32 next = i + 1 < N ? old.w[(i + 1) % N] : 0;
    const u32 from = M > 0 ? (i + M < N ? old.w[(i + M) % N] : old.w[i]) : (old.w[i] >> 16 | next << 16);
    const u32 stay = old.w[i];
    r.w[i] = on ? from : stay;
  }
  if constexpr (K > 1) move_bits<T, W, K / 2>(r, d);
}
// ... by d < W.  The empty asm keeps d's bits from being held as lane masks across
// an unrolled loop, whose scalar registers they would use up.
template <class T, int W>
__device__ __forceinline__ void move_down(Raw<T, W>& r, u32 d) {
  if (d == 0) return;
  asm volatile("" : "+v"(d));
  move_bits<T, W, W / 2>(r, d);
}

template <class T, int W>
__device__ __forceinline__ void widen(const Raw<T, W>& r, float* o) {
#pragma unroll
  for (int j = 0; j < W; ++j) {
    if constexpr (T::bytes == 4) {
      o[j] = __uint_as_float(r.w[j]);
    } else {
      const u32 w = r.w[j / 2];
      if constexpr (std::is_same<T, BF16>::value)
        o[j] = __uint_as_float(j % 2 ? (w & 0xffff0000u) : (w << 16));
      else
        o[j] = (float)__builtin_bit_cast(_Float16, (uint16_t)(j % 2 ? w >> 16 : w));
    }
  }
}

// one element, of a type known when the kernel runs
__device__ __forceinline__ float load_one(const char* p, int type) {
  if (type == ZERO_F32) return *reinterpret_cast<const float*>(p);
  const u32 h = *reinterpret_cast<const uint16_t*>(p);
  return type == ZERO_BF16 ? __uint_as_float(h << 16) : (float)__builtin_bit_cast(_Float16, (uint16_t)h);
}

// An fp32 result in the bits of its type.  The compiler would merge the conversion to
// fp16 with a product before it into one instruction that rounds once, but only in some
// of the unrolled copies, so that a value's last bit hung on its place in the tensor; the
// empty asm hides the product.
template <class T>
__device__ __forceinline__ u32 bits_of(float v) {
  if constexpr (T::bytes == 4) return __float_as_uint(v);
  else if constexpr (std::is_same<T, BF16>::value) return __builtin_bit_cast(uint16_t, (__bf16)v);
  else {
    asm("" : "+v"(v));
    return __builtin_bit_cast(uint16_t, (_Float16)v);
  }
}

__device__ __forceinline__ void store_one(char* p, int type, float v) {
  if (type == ZERO_F32) *reinterpret_cast<float*>(p) = v;
  else *reinterpret_cast<uint16_t*>(p) = (uint16_t)(type == ZERO_BF16 ? bits_of<BF16>(v) : bits_of<F16>(v));
}
__device__ __forceinline__ int one_bytes(int type) { return type == ZERO_F32 ? 4 : 2; }

template <class T, int W>
__device__ __forceinline__ void store_n(char* p, const float* v, u32 n) {
  constexpr int N = W * T::bytes / 4;
  if (n >= W) {
    u32 x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (T::bytes == 4) x[i] = bits_of<T>(v[i]);
      else x[i] = bits_of<T>(v[2 * i]) | bits_of<T>(v[2 * i + 1]) << 16;
    }
    if constexpr (N == 2) {
      const vec2 q = {x[0], x[1]};
      __builtin_nontemporal_store(q, reinterpret_cast<vec2_any*>(p));
    } else {
      const vec4 q = {x[0], x[1], x[2], x[3]};
      __builtin_nontemporal_store(q, reinterpret_cast<vec4_any*>(p));
    }
  } else {
#pragma unroll
    for (u32 j = 0; j < W; ++j) {
      if (j >= n) continue;
      if constexpr (T::bytes == 4) reinterpret_cast<float*>(p)[j] = v[j];
      else reinterpret_cast<uint16_t*>(p)[j] = (uint16_t)bits_of<T>(v[j]);
    }
  }
}

__device__ __forceinline__ u32 quotient(u32 n, const FastDiv& f) { return (u32)(((u64)n * f.m) >> f.sh); }

int launched(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e == hipSuccess) return ZERO_OK;
  char buf[256];
  snprintf(buf, sizeof buf, "%s: HIP error %d (%s)", what, (int)e, hipGetErrorString(e));
  return fail(ZERO_EHIP, buf);
}

}  // namespace
}  // namespace zk
