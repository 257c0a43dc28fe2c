// HIP kernels for gfx950 (CDNA4): the gated feed-forward block's two projections with
// the activation and the product in one kernel, and the products of its backward pass.
#include <algorithm>

#include "held.h"

namespace zk {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// The kernel's first argument, read again where this stands: fields that only the end of
// a kernel needs are not held in scalar registers through its loop.
template <class L>
__device__ __forceinline__ const L& argument() {
  auto p = (const __attribute__((address_space(4))) char*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const L*)(const __attribute__((address_space(4))) L*)p;
}

// A result's four values of consecutive columns c .. c + 3 in row r; n of them exist.
template <class T, Product KIND>
__device__ __forceinline__ void finish4(const ProductLaunch& a, int which, int64_t r, int64_t c, const float v[4], u32 n) {
  if constexpr (KIND == kInput) {
    store4<T>(a.out[0] + r * a.ld_out[0] + c * T::bytes, v, n);
  } else {
    char* const p = a.out[which] + r * a.ld_out[which] + c * one_bytes(a.out_type);
    float s[4];
#pragma unroll
    for (u32 j = 0; j < 4; ++j) {
      s[j] = v[j];
      if (a.accumulate && j < n) s[j] += load_one(p + j * one_bytes(a.out_type), a.out_type);
    }
    store4_as(p, a.out_type, s, n);
  }
}

// The same of the forward pass: gate and up.
template <class T>
__device__ __forceinline__ void finish_gated4(const ProductLaunch& a, int64_t r, int64_t c, const float g[4], const float u[4],
                                              u32 n) {
  float v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    v[j] = g[j] * (a.act == kSilu ? gate_of<kSilu>(g[j]).p : gate_of<kGelu>(g[j]).p) * u[j];
  store4<T>(a.out[0] + r * a.ld_out[0] + c * T::bytes, v, n);
  if (a.kept[0]) {
    store4<T>(a.kept[0] + r * a.ld_kept[0] + c * T::bytes, g, n);
    store4<T>(a.kept[1] + r * a.ld_kept[1] + c * T::bytes, u, n);
  }
}

// ---------------------------------------------------------------------------
// every type, size, stride and alignment
// ---------------------------------------------------------------------------

// Tiles of 64 x 64 results (of gate and of up), 32 of k at a time through registers into
// LDS as [row or column][k]; four waves of 32 x 32.
constexpr int kT = 64, kK = 32;

template <class T>
__device__ __forceinline__ void clear_raw(Raw8<T>& r, u32 n) {
  if (n >= 8) return;
  asm volatile("" : "+v"(n));
#pragma unroll
  for (u32 i = 0; i < 2 * T::bytes; ++i) {
    if constexpr (T::bytes == 4) r.w[i] = i < n ? r.w[i] : 0;
    else r.w[i] = 2 * i + 1 < n ? r.w[i] : 2 * i < n ? r.w[i] & 0xffffu : 0;
  }
}

template <class T>
struct Tile {
  static constexpr int pitch = kK * T::bytes + 16;  // bytes: rows begin in different banks
  char b[kT * pitch];
};

// Elements of one operand: [kT, kK] at (i0, k0) of a matrix whose rows are i (BY_K) or k.
template <class T, bool BY_K>
__device__ __forceinline__ void fetch(const char* p, const char* end, int64_t ld, int64_t i0, int64_t ni, int64_t k0, int64_t nk,
                                      Raw8<T>& r) {
  const u32 t = threadIdx.x;
  const int64_t row = BY_K ? i0 + t / 4 : k0 + t / 8, col = BY_K ? k0 + t % 4 * 8 : i0 + t % 8 * 8;
  const int64_t rows = BY_K ? ni : nk, cols = BY_K ? nk : ni;
  const u32 n = row < rows && col < cols ? (u32)min(cols - col, (int64_t)8) : 0;
  load8<T>(p + row * ld + col * T::bytes, end, n, r);
  clear_raw<T>(r, n);
}
template <class T, bool BY_K>
__device__ __forceinline__ void place(Tile<T>& s, const Raw8<T>& r) {
  const u32 t = threadIdx.x;
  if constexpr (BY_K) {
    vec4* const d = reinterpret_cast<vec4*>(s.b + t / 4 * Tile<T>::pitch + t % 4 * 8 * T::bytes);
#pragma unroll
    for (int i = 0; i < T::bytes / 2; ++i) d[i] = vec4{r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]};
  } else {
    const u32 k = t / 8, i0 = t % 8 * 8;
#pragma unroll
    for (u32 j = 0; j < 8; ++j) {
      char* const d = s.b + (i0 + j) * Tile<T>::pitch + k * T::bytes;
      if constexpr (T::bytes == 4) *reinterpret_cast<u32*>(d) = r.w[j];
      else *reinterpret_cast<uint16_t*>(d) = (uint16_t)(j % 2 ? r.w[j / 2] >> 16 : r.w[j / 2]);
    }
  }
}

// acc += P (16 columns at i) x Q (16 rows at j): lane l holds column 4 (l / 16) + 0 .. 3 of row l % 16.
template <class T>
__device__ __forceinline__ void multiply(const Tile<T>& p, u32 i, const Tile<T>& q, u32 j, f32x4& acc) {
  const u32 lane = threadIdx.x & 63;
  const char* const x = p.b + (i + lane % 16) * Tile<T>::pitch;
  const char* const y = q.b + (j + lane % 16) * Tile<T>::pitch;
  if constexpr (T::bytes == 4) {
#pragma unroll
    for (u32 k = 0; k < kK; k += 4)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(reinterpret_cast<const float*>(x)[k + lane / 16],
                                                 reinterpret_cast<const float*>(y)[k + lane / 16], acc, 0, 0, 0);
  } else if constexpr (std::is_same<T, BF16>::value) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(reinterpret_cast<const bf16x8*>(x)[lane / 16],
                                                  reinterpret_cast<const bf16x8*>(y)[lane / 16], acc, 0, 0, 0);
  } else {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(reinterpret_cast<const f16x8*>(x)[lane / 16],
                                                 reinterpret_cast<const f16x8*>(y)[lane / 16], acc, 0, 0, 0);
  }
}

template <class T, Product KIND>
__global__ __launch_bounds__(256) void product_kernel(const ProductLaunch a, int64_t tiles, int64_t across) {
  constexpr int NP = KIND == kForward ? 2 : 1;
  constexpr bool kQByK = KIND != kWeight, kPByK = KIND == kForward;
  __shared__ __attribute__((aligned(16))) Tile<T> sq, sp[NP];
  const u32 lane = threadIdx.x & 63, wave = threadIdx.x / 64;
  const u32 wc = wave % 2 * 32, wr = wave / 2 * 32;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int which = KIND == kWeight && tile >= tiles / 2;
    const int64_t at = which ? tile - tiles / 2 : tile;
    const int64_t r0 = at / across * kT, c0 = at % across * kT;
    f32x4 acc[NP][2][2] = {};
    Raw8<T> rq, rp[NP];
    const int64_t steps = (a.k + kK - 1) / kK, all = KIND == kInput ? 2 * steps : steps;
    auto get = [&](int64_t s) {
      const ProductLaunch& b = KIND == kInput ? argument<ProductLaunch>() : a;
      const int part = KIND == kInput ? s >= steps : which;
      const int64_t k0 = (KIND == kInput && part ? s - steps : s) * kK;
      fetch<T, kQByK>(b.q[KIND == kForward ? 0 : part], b.q_end[KIND == kForward ? 0 : part], b.ld_q[KIND == kForward ? 0 : part],
                      r0, b.rows, k0, b.k, rq);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int x = KIND == kForward ? i : KIND == kInput ? part : 0;
        fetch<T, kPByK>(b.p[x], b.p_end[x], b.ld_p[x], c0, b.cols, k0, b.k, rp[i]);
      }
    };
    get(0);
    for (int64_t s = 0; s < all; ++s) {
      __syncthreads();
      place<T, kQByK>(sq, rq);
#pragma unroll
      for (int i = 0; i < NP; ++i) place<T, kPByK>(sp[i], rp[i]);
      __syncthreads();
      if (s + 1 < all) get(s + 1);
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int y = 0; y < 2; ++y) multiply<T>(sp[i], wc + 16 * x, sq, wr + 16 * y, acc[i][x][y]);
    }
    const ProductLaunch& b = argument<ProductLaunch>();
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int64_t r = r0 + wr + 16 * y + lane % 16;
      if constexpr (KIND == kForward) {
        if (b.held[0].codes) {  // the wave has one block of every row
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            u32 top = 0;
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int j = 0; j < 4; ++j) top = max(top, finite_magnitude(acc[i][x][y][j]));
            top = max(top, (u32)__shfl_xor((int)top, 16, 64));
            top = max(top, (u32)__shfl_xor((int)top, 32, 64));
            const u32 scale = scale_of(top);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int64_t c = c0 + wc + 16 * x + lane / 16 * 4;
              if (r >= b.rows || c >= b.cols) continue;
              const float v[4] = {acc[i][x][y][0], acc[i][x][y][1], acc[i][x][y][2], acc[i][x][y][3]};
              store_codes4(b.held[i], r, c, v, scale, (u32)min(b.cols - c, (int64_t)4));
              if (c % kBlock == 0) b.held[i].scales[r * b.held[i].ld_scales + c / kBlock] = (char)scale;
            }
          }
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int64_t c = c0 + wc + 16 * x + lane / 16 * 4;
        if (r >= b.rows || c >= b.cols) continue;
        const u32 n = (u32)min(b.cols - c, (int64_t)4);
        const float v[4] = {acc[0][x][y][0], acc[0][x][y][1], acc[0][x][y][2], acc[0][x][y][3]};
        if constexpr (KIND == kForward) {
          const float u[4] = {acc[1][x][y][0], acc[1][x][y][1], acc[1][x][y][2], acc[1][x][y][3]};
          finish_gated4<T>(b, r, c, v, u, n);
        } else {
          finish4<T, KIND>(b, which, r, c, v, n);
        }
      }
    }
  }
}

template <class T, Product KIND>
int product_as(const ProductLaunch& a, hipStream_t s) {
  const int64_t across = (a.cols + kT - 1) / kT;
  const int64_t tiles = (a.rows + kT - 1) / kT * across * (KIND == kWeight ? 2 : 1);
  hipLaunchKernelGGL((product_kernel<T, KIND>), dim3((u32)std::min<int64_t>(tiles, kMaxGroups)), dim3(256), 0, s, a, tiles,
                     across);
  return launched(KIND == kForward ? "gated projections" : KIND == kInput ? "gated input gradient" : "gated weight gradient");
}

template <Product KIND>
int product_of(const ProductLaunch& a, zero_dtype_t t, hipStream_t s) {
  switch (t) {
    case ZERO_F32: return product_as<F32, KIND>(a, s);
    case ZERO_BF16: return product_as<BF16, KIND>(a, s);
    default: return product_as<F16, KIND>(a, s);
  }
}

}  // namespace

int64_t product_ws_bytes(int64_t, int64_t, int64_t) { return 0; }

int launch_product(Product kind, const ProductLaunch& a, zero_dtype_t t, void* stream) {
  switch (kind) {
    case kForward: return product_of<kForward>(a, t, (hipStream_t)stream);
    case kInput: return product_of<kInput>(a, t, (hipStream_t)stream);
    default: return product_of<kWeight>(a, t, (hipStream_t)stream);
  }
}

}  // namespace zk
