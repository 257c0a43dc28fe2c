// Device code shared by the feed-forward sub-layer's kernels: 8 columns of a row at
// a time, matrices held in 8 bits, the gated activation.  Included inside a kernel
// source only.
#pragma once

#include "elements.h"
#include "layer.h"

namespace zk {
namespace {

typedef vec2 vec2_byte __attribute__((aligned(1)));  // at any address
typedef vec4 vec4_byte __attribute__((aligned(1)));

typedef u32 u32_byte __attribute__((aligned(1)));
typedef uint16_t u16_byte __attribute__((aligned(1)));

// The kernel's first argument, read again where this stands: fields that only the end of
// a kernel needs are not held in scalar registers through its loop.
template <class L>
__device__ __forceinline__ const L& argument() {
  auto p = (const __attribute__((address_space(4))) char*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const L*)(const __attribute__((address_space(4))) L*)p;
}

// 8 elements of a row, raw
template <class T>
struct Raw8 {
  u32 w[2 * T::bytes];
};

// The n <= 8 elements at p that exist in the row; behind them anything.  Vectors where
// 8 elements lie before `end`, the end of the tensor, else (its last few
// elements, and tensors shorter than 8) one by one.
// `inside`: a whole wave's answer that every vector lies before the end.
template <class T>
__device__ __forceinline__ void load8(const char* p, const char* end, u32 n, Raw8<T>& r, bool inside = false) {
#pragma unroll
  for (int i = 0; i < 2 * T::bytes; ++i) r.w[i] = 0;
  if (n == 0) return;
  if (inside || end - p >= 8 * T::bytes) {
#pragma unroll
    for (int i = 0; i < T::bytes / 2; ++i) {
      const vec4 q = reinterpret_cast<const vec4_any*>(p)[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) r.w[4 * i + j] = q[j];
    }
  } else {
#pragma unroll 1
    for (u32 j = 0; j < n; ++j) {
      u32 e;
      if constexpr (T::bytes == 4) e = reinterpret_cast<const u32*>(p)[j];
      else e = (u32)reinterpret_cast<const uint16_t*>(p)[j] << (16 * (j % 2));
#pragma unroll
      for (u32 i = 0; i < 2 * T::bytes; ++i) r.w[i] |= i == j * T::bytes / 4 ? e : 0;
    }
  }
}

// Zeros behind the n-th value.  The empty asm keeps the comparisons' lane masks from
// being held across an unrolled loop, whose scalar registers they would use up.
__device__ __forceinline__ void clear_tail(float v[8], u32 n) {
  if (n >= 8) return;
  asm volatile("" : "+v"(n));
#pragma unroll
  for (u32 j = 0; j < 8; ++j) v[j] = j < n ? v[j] : 0.0f;
}

// the values in fp32, zeros behind the n-th
template <class T>
__device__ __forceinline__ void values8(const Raw8<T>& r, u32 n, float v[8]) {
  Raw<T, 8> x;
#pragma unroll
  for (int i = 0; i < 2 * T::bytes; ++i) x.w[i] = r.w[i];
  widen<T, 8>(x, v);
  clear_tail(v, n);
}

// The first n of 4 elements at p, of a type known when the kernel runs; zeros behind them.
__device__ __forceinline__ void load4_as(const char* p, int type, u32 n, float v[4]) {
  if (n < 4) {
#pragma unroll
    for (u32 j = 0; j < 4; ++j) v[j] = j < n ? load_one(p + j * one_bytes(type), type) : 0.0f;
  } else if (type == ZERO_F32) {
    const vec4 q = *reinterpret_cast<const vec4_any*>(p);
    const Raw<F32, 4> r = {{q[0], q[1], q[2], q[3]}};
    widen<F32, 4>(r, v);
  } else {
    const vec2 q = *reinterpret_cast<const vec2_any*>(p);
    if (type == ZERO_BF16) widen<BF16, 4>(Raw<BF16, 4>{{q[0], q[1]}}, v);
    else widen<F16, 4>(Raw<F16, 4>{{q[0], q[1]}}, v);
  }
}

// The first n < 2 K elements of the N words w, by the bits K, K / 2 .. 1 of n.
template <int BYTES, int K, int N>
__device__ __forceinline__ void store_bits(char* p, u32 (&w)[N], u32 n) {
  constexpr int M = K * BYTES / 4;  // words of K elements; 0: less than one
  if (n & K) {
    if constexpr (K * BYTES == 16) {
      const vec4 q = {w[0], w[1], w[2], w[3]};
      *reinterpret_cast<vec4_any*>(p) = q;
    } else if constexpr (K * BYTES == 8) {
      const vec2 q = {w[0], w[1]};
      *reinterpret_cast<vec2_any*>(p) = q;
    } else if constexpr (K * BYTES == 4) {
      *reinterpret_cast<u32_byte*>(p) = w[0];
    } else if constexpr (K * BYTES == 2) {
      *reinterpret_cast<u16_byte*>(p) = (uint16_t)w[0];
    } else {
      *p = (char)w[0];
    }
    p += K * BYTES;
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = M > 0 ? (i + M < N ? w[(i + M) % N] : 0) : w[i] >> (K * BYTES * 8 % 32);
  }
  if constexpr (K > 1) store_bits<BYTES, K / 2>(p, w, n);
}

// 8 values rounded to a type
template <class T>
__device__ __forceinline__ Raw8<T> round8(const float v[8]) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < 2 * T::bytes; ++i) {
    if constexpr (T::bytes == 4) r.w[i] = bits_of<T>(v[i]);
    else r.w[i] = bits_of<T>(v[2 * i]) | bits_of<T>(v[2 * i + 1]) << 16;
  }
  return r;
}

// Stores n <= 8 values, not to be read again soon.
template <class T>
__device__ __forceinline__ void store8(char* p, const Raw8<T>& r, u32 n) {
  constexpr int N = 2 * T::bytes;
  u32 w[N];
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = r.w[i];
  if (n == 8) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const vec4 q = {w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
      __builtin_nontemporal_store(q, reinterpret_cast<vec4_any*>(p) + i);
    }
  } else {
    asm volatile("" : "+v"(n));
    store_bits<T::bytes, 4>(p, w, n);
  }
}

template <class T>
__device__ __forceinline__ void store8(char* p, const float v[8], u32 n) {
  store8<T>(p, round8<T>(v), n);
}

// Stores the first n of 4 values.
template <class T>
__device__ __forceinline__ void store4(char* p, const float v[4], u32 n) {
  constexpr int N = T::bytes;
  u32 w[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (T::bytes == 4) w[i] = bits_of<T>(v[i]);
    else w[i] = bits_of<T>(v[2 * i]) | bits_of<T>(v[2 * i + 1]) << 16;
  }
  if (n >= 4) {
    if constexpr (N == 4) {
      const vec4 q = {w[0], w[1], w[2], w[3]};
      *reinterpret_cast<vec4_any*>(p) = q;
    } else {
      const vec2 q = {w[0], w[1]};
      *reinterpret_cast<vec2_any*>(p) = q;
    }
  } else {
    store_bits<T::bytes, 2>(p, w, n);
  }
}
__device__ __forceinline__ void store4_as(char* p, int type, const float v[4], u32 n) {
  if (type == ZERO_F32) store4<F32>(p, v, n);
  else if (type == ZERO_BF16) store4<BF16>(p, v, n);
  else store4<F16>(p, v, n);
}

// The same of a type known when the kernel runs.
__device__ __forceinline__ void store8_as(char* p, int type, const float v[8], u32 n) {
  if (type == ZERO_F32) store8<F32>(p, v, n);
  else if (type == ZERO_BF16) store8<BF16>(p, v, n);
  else store8<F16>(p, v, n);
}
__device__ __forceinline__ void load8_as(const char* p, const char* end, int type, u32 n, Raw8<F32>& r) {
  if (type == ZERO_F32) {
    load8<F32>(p, end, n, r);
  } else {
    Raw8<BF16> q;
    load8<BF16>(p, end, n, q);
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = q.w[i];
  }
}
__device__ __forceinline__ void values8_as(const Raw8<F32>& r, int type, u32 n, float v[8]) {
  if (type == ZERO_F32) {
    values8<F32>(r, n, v);
  } else if (type == ZERO_BF16) {
    values8<BF16>(Raw8<BF16>{r.w[0], r.w[1], r.w[2], r.w[3]}, n, v);
  } else {
    values8<F16>(Raw8<F16>{r.w[0], r.w[1], r.w[2], r.w[3]}, n, v);
  }
}

// ---------------------------------------------------------------------------
// 8 bits
// ---------------------------------------------------------------------------

// The scale byte of a block whose largest finite magnitude has these fp32 bits: the
// smallest power of two, from 2^-127 up, that brings it to at most 448 = 1.75 * 2^8.
__device__ __forceinline__ u32 scale_of(u32 top) {
  const u32 s = (top >> 23) + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
  return s > 8 ? s - 8 : 0;
}
// 1 / scale, exact
__device__ __forceinline__ float inverse_scale(u32 s) { return __uint_as_float((254 - s) << 23); }
// the scale; 2^-127 (byte 0) is a subnormal, and 255 is e8m0's NaN: both have the fraction's first bit set
__device__ __forceinline__ float scale_value(u32 s) {
  return __uint_as_float(s << 23 | (((s + 1) & 254) == 0 ? 0x400000u : 0));
}

__device__ __forceinline__ bool finite_bits(u32 b) { return (b & 0x7fffffffu) < 0x7f800000u; }

// Infinities and NaN do not count towards the scale, so that they spoil no other value.
__device__ __forceinline__ u32 finite_magnitude(float v) {
  const u32 b = __float_as_uint(v);
  return finite_bits(b) ? b & 0x7fffffffu : 0;
}
// e4m3 has no infinity: NaN stands for both
__device__ __forceinline__ float held_input(float v) {
  return finite_bits(__float_as_uint(v)) ? v : __uint_as_float(0x7fc00000u);
}
// Four codes of values that are finite or NaN.  The conversion rounds to nearest, ties to even, and nothing is past 448.
__device__ __forceinline__ u32 codes4_finite(const float* v, float inv) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inv, v[1] * inv, 0, false);
  return (u32)__builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inv, v[3] * inv, w, true);
}
// Four codes of any values.
__device__ __forceinline__ u32 codes4(const float* v, float inv) {
  const float f[4] = {held_input(v[0]), held_input(v[1]), held_input(v[2]), held_input(v[3])};
  return codes4_finite(f, inv);
}

// Holds 8 columns of a row; the four lanes of a quad have one block's 32 columns, and
// all of them take part.  Values behind the n-th are zeros.
__device__ __forceinline__ void hold8(const Held& h, int64_t row, u32 group, const float x[8], u32 n) {
  u32 top = 0;
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = x[j];
    top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
  }
  if (__builtin_amdgcn_ballot_w64(top >= 0x7f800000u)) {  // infinities and NaN
    top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      top = max(top, finite_magnitude(v[j]));
      v[j] = held_input(v[j]);
    }
  }
  top = max(top, (u32)__builtin_amdgcn_mov_dpp((int)top, 0xB1, 0xF, 0xF, true));  // quad_perm [1, 0, 3, 2]
  top = max(top, (u32)__builtin_amdgcn_mov_dpp((int)top, 0x4E, 0xF, 0xF, true));  // quad_perm [2, 3, 0, 1]
  if (n == 0) return;
  const u32 s = scale_of(top);
  const float inv = inverse_scale(s);
  const u32 lo = codes4_finite(v, inv), hi = codes4_finite(v + 4, inv);
  char* p = h.codes + row * h.ld_codes + (int64_t)group * 8;
  if (n == 8) {
    const vec2 q = {lo, hi};
    __builtin_nontemporal_store(q, reinterpret_cast<vec2_byte*>(p));
  } else {
    u32 w[2] = {lo, hi}, k = n;
    asm volatile("" : "+v"(k));
    store_bits<1, 4>(p, w, k);
  }
  if (group % 4 == 0) h.scales[row * h.ld_scales + group / 4] = (char)s;
}

// 8 columns of a row held in 8 bits, raw
struct RawHeld {
  u32 lo, hi, scale;
};
__device__ __forceinline__ void load_held(const Held& h, int64_t row, u32 group, u32 n, RawHeld& r, bool inside = false) {
  r.lo = r.hi = r.scale = 0;
  if (n == 0) return;
  const char* p = h.codes + row * h.ld_codes + (int64_t)group * 8;
  if (inside || h.codes_end - p >= 8) {
    const vec2 q = *reinterpret_cast<const vec2_byte*>(p);
    r.lo = q.x;
    r.hi = q.y;
  } else {
#pragma unroll 1
    for (u32 j = 0; j < n; ++j) {
      const u32 b = (u32)(uint8_t)p[j] << (8 * (j % 4));
      r.lo |= j < 4 ? b : 0;
      r.hi |= j < 4 ? 0 : b;
    }
  }
  r.scale = (uint8_t)h.scales[row * h.ld_scales + group / 4];
}
__device__ __forceinline__ void held_values(const RawHeld& r, u32 n, float v[8]) {
  const float s = scale_value(r.scale);
  typedef float f2 __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const u32 w = i < 2 ? r.lo : r.hi;
    const f2 q = i % 2 ? __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true) : __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    v[2 * i] = q.x * s;
    v[2 * i + 1] = q.y * s;
  }
  clear_tail(v, n);
}

// Holds 4 columns of a row from `col` on, a multiple of 4, with the block's scale byte.
__device__ __forceinline__ void store_codes4(const Held& h, int64_t row, int64_t col, const float v[4], u32 s, u32 n) {
  u32 w[1] = {codes4(v, inverse_scale(s))};
  char* const p = h.codes + row * h.ld_codes + col;
  if (n >= 4) *reinterpret_cast<u32_byte*>(p) = w[0];
  else store_bits<1, 2>(p, w, n);
}

// ---------------------------------------------------------------------------
// sums over the lanes of a wave: every lane gets the same bits
// ---------------------------------------------------------------------------

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float((u32)__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const u64 b = __builtin_bit_cast(u64, v);
  const u32 lo = (u32)__builtin_amdgcn_mov_dpp((int)(u32)b, CTRL, 0xF, 0xF, true);
  const u32 hi = (u32)__builtin_amdgcn_mov_dpp((int)(u32)(b >> 32), CTRL, 0xF, 0xF, true);
  return __builtin_bit_cast(double, (u64)hi << 32 | lo);
}
template <class S>
__device__ __forceinline__ S wave_sum(S v) {
  v += dpp<0xB1>(v);   // the other lane of the pair
  v += dpp<0x4E>(v);   // the other pair of four
  v += dpp<0x141>(v);  // the other four of eight (row_half_mirror)
  v += dpp<0x140>(v);  // the other eight of sixteen (row_mirror)
  v += __shfl_xor(v, 16, 64);
  v += __shfl_xor(v, 32, 64);
  return v;
}

// ---------------------------------------------------------------------------
// the gate
// ---------------------------------------------------------------------------

// act(g) = g * p, act'(g) = p + g * p * q * slope, with p a logistic function and q = 1 - p:
//   SiLU            p = 1 / (1 + exp(-z)), z = g
//   GELU, tanh form p = (1 + tanh(z / 2)) / 2 = 1 / (1 + exp(-z)), z = 2 sqrt(2 / pi) (g + 0.044715 g^3)
struct Gate {
  float p, q, slope;
};
constexpr double kGeluScale = 1.59576912160573071, kGeluCube = 0.044715;  // 2 sqrt(2 / pi)

// For results of 16 bits: the hardware's exp2 and reciprocal, each within an ulp or so, of an argument of fp32,
// whose rounding alone puts p off by some 2^-23 |z| of itself (4e-6 at 60, of half a step of 2e-3 or 5e-4), and 0
// below 2^-126.
template <int ACT>
__device__ __forceinline__ Gate gate_16(float g) {
  constexpr float k2 = (float)kGeluScale, c = (float)kGeluCube;
  const float g2 = fminf(g * g, 1e30f);  // beyond, p is 0 or 1 and the slope only has to stay finite
  const float z = ACT == kSilu ? g : k2 * g * __builtin_fmaf(c, g2, 1.0f);
  const float p = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504088896340736f));
  return Gate{p, 1.0f - p, ACT == kSilu ? 1.0f : k2 * __builtin_fmaf(3.0f * c, g2, 1.0f)};
}

// For fp32 results: from t = exp(-|z|), so that both p and q keep their digits, down to the subnormals; GELU's z is
// computed in fp64, since exp turns its absolute error into a relative one.  p and q are good to some 3e-7 of themselves;
// gate_16's would be off by 3e-6 at z = -50, for up to 1% less time where matrices are large (gradient of 2048 x 14336,
// GELU from 8 bits, 138 us and 139; forward pass of 1024 tokens, 2048 x 5504, 384 and 388), 2 to 5% where sums are short
// (4096 tokens, 512 x 1376, 104 and 107, GELU 108; 8192, 256 x 1376, 106 and 110, GELU 114).
template <int ACT>
__device__ __forceinline__ Gate gate_32(float g) {
  float z = g, rest = 0.0f, slope = 1.0f;  // z + rest
  if constexpr (ACT == kGelu) {
    const double d = g, w = fmin(fmax(kGeluScale * d * __builtin_fma(kGeluCube * d, d, 1.0), -256.0), 256.0);
    z = (float)w;
    rest = (float)(w - (double)z);
    const float g2 = fminf(g * g, 1e30f);  // beyond, p or q is 0 and the slope only has to stay finite
    slope = (float)kGeluScale * __builtin_fmaf(3.0f * (float)kGeluCube, g2, 1.0f);
  }
  // exp(-|z|) = 2^n 2^f with n whole and |f| <= 1/2; log2(e) in two parts, so that f is off by 2^-25 at most
  constexpr double kLog2e = 1.44269504088896340736;
  constexpr float kHigh = (float)kLog2e, kLow = (float)(kLog2e - (double)kHigh);
  const float m = fminf(fabsf(z), 256.0f);  // exp(-256) is 0
  const float n = __builtin_rintf(m * -kHigh);
  float f = __builtin_fmaf(m, -kLow, __builtin_fmaf(m, -kHigh, -n));
  if constexpr (ACT == kGelu) f = __builtin_fmaf(z < 0.0f ? rest : -rest, kHigh, f);
  const float t = __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
  // 1 / (1 + t): the hardware's estimate and one of Newton's steps
  const float sum = 1.0f + t, near = __builtin_amdgcn_rcpf(sum);
  const float large = __builtin_fmaf(__builtin_fmaf(-sum, near, 1.0f), near, near), small = t * large;
  return z < 0.0f ? Gate{small, large, slope} : Gate{large, small, slope};
}

// T: the results' type
template <class T, int ACT>
__device__ __forceinline__ Gate gate_of(float g) {
  if constexpr (T::bytes == 4) return gate_32<ACT>(g);
  else return gate_16<ACT>(g);
}

}  // namespace
}  // namespace zk
