// HIP kernels for gfx950 (CDNA4): the gated feed-forward block's two projections with
// the activation and the product in one kernel, and the products of its backward pass.
#include <algorithm>

#include "held.h"

namespace zk {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// A result's four values of consecutive columns c .. c + 3 in row r; n of them exist.
template <class T, Product KIND>
__device__ __forceinline__ void finish4(const ProductLaunch& a, int which, int64_t r, int64_t c, const float v[4], u32 n) {
  if constexpr (KIND == kInput) {
    store4<T>(a.out[0] + r * a.ld_out[0] + c * T::bytes, v, n);
  } else {
    char* const p = a.out[which] + r * a.ld_out[which] + c * one_bytes(a.out_type);
    float s[4] = {v[0], v[1], v[2], v[3]};
    if (a.accumulate) {
      float old[4];
      load4_as(p, a.out_type, n, old);
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] += old[j];
    }
    store4_as(p, a.out_type, s, n);
  }
}

__device__ __forceinline__ float gated_value(int32_t act, float g, float u) {
  return g * (act == kSilu ? gate_of<kSilu>(g).p : gate_of<kGelu>(g).p) * u;
}

// The same of the forward pass: gate and up.
template <class T>
__device__ __forceinline__ void finish_gated4(const ProductLaunch& a, int64_t r, int64_t c, const float g[4], const float u[4],
                                              u32 n) {
  float v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = gated_value(a.act, g[j], u[j]);
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

// ---------------------------------------------------------------------------
// results by way of LDS
// ---------------------------------------------------------------------------

// 32 rows of a wave, each of WIDE 16-bit results, 32 fp32 ones or WIDE codes, 16 bytes apart from the next
// row so that the lanes' rows begin in different banks.  In a block of 32 x 32 results lane l
// has row l % 32, columns 8 j + 4 (l / 32) + 0 .. 3.
constexpr u32 kStageBytes = 32 * 144;

template <class T, int WIDE>
__device__ __forceinline__ void stage_bits(char* s, u32 col, const float v[4]) {
  const u32 lane = threadIdx.x & 63;
  const vec2 w = {bits_of<T>(v[0]) | bits_of<T>(v[1]) << 16, bits_of<T>(v[2]) | bits_of<T>(v[3]) << 16};
  *reinterpret_cast<vec2*>(s + lane % 32 * (WIDE * 2 + 16) + (col + lane / 32 * 4) * 2) = w;
}
// Writes what is staged to rows from r on, columns from c on.
template <class T, int WIDE>
__device__ __forceinline__ void flush_bits(const char* s, char* out, int64_t ld, int64_t r, int64_t rows, int64_t c,
                                           int64_t cols) {
  constexpr u32 kLanes = WIDE / 8;  // of a row
  const u32 lane = threadIdx.x & 63;
  const int64_t col = c + lane % kLanes * 8;
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (u32 i = 0; i < 32; i += 64 / kLanes) {
    const u32 row = i + lane / kLanes;
    const vec4 q = *reinterpret_cast<const vec4*>(s + row * (WIDE * 2 + 16) + lane % kLanes * 16);
    if (r + row >= rows || col >= cols) continue;
    char* const p = out + (r + row) * ld + col * T::bytes;
    const u32 n = (u32)min(cols - col, (int64_t)8);
    if (n == 8) {
      *reinterpret_cast<vec4_any*>(p) = q;
    } else {
      u32 w[4] = {q[0], q[1], q[2], q[3]};
      store_bits<T::bytes, 4>(p, w, n);
    }
  }
  __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ void stage_floats(char* s, u32 col, f32x4 v) {
  const u32 lane = threadIdx.x & 63;
  *reinterpret_cast<f32x4*>(s + lane % 32 * 144 + (col + lane / 32 * 4) * 4) = v;
}
// The weight gradient's results, added to what is there where asked.
__device__ __forceinline__ void flush_floats(const char* s, const ProductLaunch& a, int which, int64_t r, int64_t c) {
  const u32 lane = threadIdx.x & 63;
  const int64_t col = c + lane % 8 * 4;
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (u32 i = 0; i < 32; i += 8) {
    const u32 row = i + lane / 8;
    const f32x4 q = *reinterpret_cast<const f32x4*>(s + row * 144 + lane % 8 * 16);
    if (r + row >= a.rows || col >= a.cols) continue;
    const float v[4] = {q[0], q[1], q[2], q[3]};
    finish4<BF16, kWeight>(a, which, r + row, col, v, (u32)min(a.cols - col, (int64_t)4));
  }
  __builtin_amdgcn_wave_barrier();
}

// A split's sums, dense, `out` at row r; cols is a multiple of 8.
__device__ __forceinline__ void flush_partial(const char* s, float* out, int64_t r, int64_t rows, int64_t c, int64_t cols) {
  const u32 lane = threadIdx.x & 63;
  const int64_t col = c + lane % 8 * 4;
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (u32 i = 0; i < 32; i += 8) {
    const u32 row = i + lane / 8;
    const f32x4 q = *reinterpret_cast<const f32x4*>(s + row * 144 + lane % 8 * 16);
    if (r + row < rows && col < cols) *reinterpret_cast<f32x4*>(out + row * cols + col) = q;
  }
  __builtin_amdgcn_wave_barrier();
}

// Stages a block's codes and stores its scales.  The block's columns begin at c, at `at` of what is staged.
template <int WIDE>
__device__ __forceinline__ void hold_block(char* s, const Held& h, const f32x16& v, int64_t r, int64_t rows, int64_t c, u32 at,
                                           int64_t cols) {
  const u32 lane = threadIdx.x & 63;
  float f[16];
  const int64_t left = cols - c - lane / 32 * 4;  // columns beyond the last hold what the tile read there
  u32 top = 0;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    f[j] = j / 4 * 8 + j % 4 < left ? v[j] : 0.0f;
    top = max(top, __float_as_uint(f[j]) & 0x7fffffffu);
  }
  if (__builtin_amdgcn_ballot_w64(top >= 0x7f800000u)) {  // infinities and NaN
    top = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      top = max(top, finite_magnitude(f[j]));
      f[j] = held_input(f[j]);
    }
  }
  top = max(top, (u32)__shfl_xor((int)top, 32, 64));
  const u32 scale = scale_of(top);
  const float inv = inverse_scale(scale);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<u32*>(s + lane % 32 * (WIDE + 16) + at + 8 * j + lane / 32 * 4) = codes4_finite(f + 4 * j, inv);
  if (lane < 32 && r + lane < rows && c < cols) h.scales[(r + lane) * h.ld_scales + c / kBlock] = (char)scale;
}
template <int WIDE>
__device__ __forceinline__ void flush_codes(const char* s, const Held& h, int64_t r, int64_t rows, int64_t c, int64_t cols) {
  constexpr u32 kLanes = WIDE / 16;
  const u32 lane = threadIdx.x & 63;
  const int64_t col = c + lane % kLanes * 16;
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (u32 i = 0; i < 32; i += 64 / kLanes) {
    const u32 row = i + lane / kLanes;
    if (row >= 32) continue;
    const vec4 q = *reinterpret_cast<const vec4*>(s + row * (WIDE + 16) + lane % kLanes * 16);
    if (r + row >= rows || col >= cols) continue;
    char* const p = h.codes + (r + row) * h.ld_codes + col;
    const u32 n = (u32)min(cols - col, (int64_t)16);
    if (n == 16) {
      *reinterpret_cast<vec4_byte*>(p) = q;
    } else {
      u32 w[4] = {q[0], q[1], q[2], q[3]};
      store_bits<1, 8>(p, w, n);
    }
  }
  __builtin_amdgcn_wave_barrier();
}

// ---------------------------------------------------------------------------
// 16-bit types at multiples of 16 bytes
// ---------------------------------------------------------------------------

// Tiles of TILE x TILE results (of gate and up in the forward pass TILE x TILE / 2 each).
// A wave has XB x 2 blocks of 32 x 32 results.  The operands' tiles go from global memory
// straight into LDS (16 bytes a lane, no registers between), two to four steps of 32 of k
// before they are used: under load a copy takes a microsecond and more, a step of matrix
// instructions 0.6.
//
// LDS holds an operand as its rows lie in memory.  Rows of k are copied 64 of k at a time,
// 128 bytes, whole lines of the L2 (with half lines its requests doubled, and the
// forward pass took 1626 us in place of FWD_US): unit (16 bytes) j of row i sits at
// j ^ (i / 2 % 8), so that the 16-byte reads of 16 lanes in neighbouring rows meet every bank once.
// Rows of the other index ([32 k][TILE]) are read transposed, 4 rows of 16 columns by 16
// lanes: unit j of row k sits at j ^ 2 (k % 4) in tiles of 128; in tiles of 256, whose kernels
// have no registers for the addresses that this takes, at j ^ 2 (k % 2), with 64 bytes
// left out before every odd pair of rows.  Either way the 4 rows lie in different banks.
// The DMA writes LDS in lane order, 1024 bytes a wave, so a lane fetches the unit that belongs
// at its place.
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef short i16x8 __attribute__((ext_vector_type(8)));
constexpr int kStep = 32;
template <bool BY_K>
constexpr int kDeep = BY_K ? 2 * kStep : kStep;  // of k, copied at a time
template <bool BY_K>
constexpr int kRounds = BY_K ? 4 : 2;            // 16 bytes a thread and round

template <int TILE>
constexpr int kTileThreads = TILE == 256 ? 512 : 256;
template <int TILE, bool BY_K>
constexpr int kTileBytes = TILE * kDeep<BY_K> * 2 + (TILE == 256 && !BY_K ? 512 : 0);
// Where the 1024 bytes of chunk c of a tile begin.
template <int TILE, bool BY_K>
__device__ __forceinline__ u32 chunk_at(u32 c) {
  return c * 1024 + (TILE == 256 && !BY_K ? (c + 1) / 2 * 64 : 0);
}
template <int TILE>
__device__ __forceinline__ u32 swizzle(u32 k) {
  return TILE == 256 ? k % 2 * 2 : k % 4 * 2;
}

// This thread's place of round q in an operand's tile: byte offset from the tile's first element.
// i0, ni: the tile's first row (column) and the matrix's number of them, beyond which the last
// ones stand in (what they give is not stored).
template <int TILE, bool BY_K>
__device__ __forceinline__ u32 place_of(int q, int64_t ld, int64_t i0, int64_t ni) {
  constexpr u32 kN = kTileThreads<TILE>;
  const u32 t = threadIdx.x;
  if constexpr (BY_K) {
    const u32 row = q * (kN / 8) + t / 8;
    return (u32)min((int64_t)row, ni - 1 - i0) * (u32)ld + ((t % 8) ^ (t / 16 % 8)) * 16;
  } else {
    constexpr u32 kUnits = TILE / 8;
    const u32 k = q * (kN / kUnits) + t / kUnits;
    const u32 col = ((t % kUnits) ^ swizzle<TILE>(k)) * 8;
    return k * (u32)ld + (u32)min((int64_t)col, ni - 8 - i0) * 2;
  }
}
// Whether it lies within the last `left` of k.
template <int TILE, bool BY_K>
__device__ __forceinline__ bool inside(int q, int left) {
  constexpr u32 kN = kTileThreads<TILE>, kUnits = TILE / 8;
  u32 t = threadIdx.x;
  asm volatile("" : "+v"(t));  // what this needs is not held in registers through the loop
  return (int)(BY_K ? ((t % 8) ^ (t / 16 % 8)) * 8 : q * (kN / kUnits) + t / kUnits) < left;
}

// What copies read from: bytes from p on, by 32-bit offsets.  A buffer descriptor costs a copy no vector
// instruction and no register for its address.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const char* p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p), 0, 0x7fffffff, 0x00020000);
}

// Starts the copy of round q.  PART: the last of k, beyond whose `left` there are zeros.
template <int TILE, bool BY_K, bool PART>
__device__ __forceinline__ void copy_place(char* lds, __amdgpu_buffer_rsrc_t from, u32 off, int q, int left) {
  constexpr u32 kN = kTileThreads<TILE>;
  char* const to = lds + chunk_at<TILE, BY_K>(q * (kN / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x / 64));
  if (!PART || inside<TILE, BY_K>(q, left)) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void*)to, 16, off, 0, 0, 0);
  } else {
    u32 t = threadIdx.x, zero = 0;
    asm volatile("" : "+v"(t), "+v"(zero));
    *reinterpret_cast<vec4*>(to + t % 64 * 16) = vec4{zero, zero, zero, zero};
  }
}

// This lane's offsets of the blocks of 32 rows (columns) from i0, i0 + 32 .. on.  The compiler has to
// see an LDS address as one sum, or it loses which tile it lies in.
template <int TILE, bool BY_K, int N>
__device__ __forceinline__ void block_offsets(u32 (&at)[N], u32 i0) {
  const u32 lane = threadIdx.x & 63;
  const u32 j = lane % 16 / 4, unit = lane % 32 / 16 * 2 + lane % 4 / 2;  // row of 4, unit of 32 columns
  constexpr bool kOne = BY_K || TILE == 256;  // the others lie a fixed way behind the first
#pragma unroll
  for (int x = 0; x < N; ++x) {
    if (kOne && x > 0) {
      at[x] = at[0] + x * (BY_K ? 32 * 128 : 64);
      continue;
    }
    const u32 i = i0 + 32 * x;
    if constexpr (BY_K) at[x] = (i + lane % 32) * 128 + ((lane / 32) ^ (lane / 2 % 8)) * 16;
    else if constexpr (TILE == 256)
      at[x] = lane / 32 * chunk_at<TILE, false>(4) + j / 2 * chunk_at<TILE, false>(1) + j % 2 * 512 + i * 2 +
              (unit ^ swizzle<TILE>(j)) * 16 + lane % 2 * 8;
    else at[x] = (lane / 32 * 8 + j) * (TILE * 2) + ((i / 8 + unit) ^ swizzle<TILE>(j)) * 16 + lane % 2 * 8;
    if constexpr (!BY_K) asm("" : "+v"(at[x]));
  }
}

// 16 of k from 16 s on of a block: lane l has row (column) l % 32, k 8 (l / 32) + 0 .. 7.
template <int TILE, bool BY_K>
__device__ __forceinline__ i16x8 fragment(const char* lds, u32 at, u32 s) {
  if constexpr (BY_K) {
    return *reinterpret_cast<const i16x8*>(lds + (at ^ (s * 32)));
  } else {
    const u32 p = at + (TILE == 256 ? chunk_at<TILE, false>(8 * s) : 16 * s * (TILE * 2));
    const u32 p4 = p + (TILE == 256 ? chunk_at<TILE, false>(2) : 4 * (TILE * 2));  // 4 rows on
    typedef __attribute__((address_space(3))) i16x4* lds_ptr;
    const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(lds + p));
    const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(lds + p4));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }
}

template <class T>
__device__ __forceinline__ f32x16 mfma32(i16x8 p, i16x8 q, f32x16 acc) {
  if constexpr (std::is_same<T, BF16>::value)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, p), __builtin_bit_cast(bf16x8, q), acc, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, p), __builtin_bit_cast(f16x8, q), acc, 0, 0, 0);
}

// All but the newest LATER copies have arrived, for every wave, and every wave's reads are done.
template <int LATER>
__device__ __forceinline__ void turn() {
  static_assert(LATER < 16, "the field's low bits");
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x70 | LATER);  // vmcnt(LATER) lgkmcnt(0), known to the compiler, which adds no others
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Orders the scheduling region: one matrix instruction, one of the copies, EACH reads of LDS, and so on.
template <int MFMA, int COPIES, int READS, int EACH>
__device__ __forceinline__ void interleave() {
  if constexpr (MFMA > 0) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (COPIES > 0) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    if constexpr (READS > 0) __builtin_amdgcn_sched_group_barrier(0x100, READS < EACH ? READS : EACH, 0);
    interleave<MFMA - 1, (COPIES > 0 ? COPIES - 1 : 0), (READS > EACH ? READS - EACH : 0), EACH>();
  }
}

// The r-th and c-th tile of workgroup b.  Workgroups go round the eight XCDs; each
// XCD takes a run of tiles of its own, down columns of `kTall` tiles, so that the
// tiles that run on it at a time share rows and columns in its L2.
constexpr u32 kTall = 4;
__device__ __forceinline__ void tile_of(u32 b, u32 down, u32 across, u32& r, u32& c) {
  const u32 n = down * across, xcd = b % 8, each = n / 8, more = n % 8;
  const u32 i = xcd * each + min(xcd, more) + b / 8;
  const u32 band = i / (kTall * across), in = i % (kTall * across);
  const u32 tall = min(kTall, down - band * kTall);
  r = band * kTall + in % tall;
  c = in / tall;
}

template <class T, Product KIND, int TILE>
__global__ __launch_bounds__(kTileThreads<TILE>) void tiled_kernel(const ProductLaunch a, u32 down, u32 across, u32 splits) {
  constexpr bool kQByK = KIND != kWeight, kPByK = KIND == kForward;
  constexpr int WC = 2, WR = TILE == 256 ? 4 : 2;
  constexpr int XB = TILE / WC / 32, YB = TILE / WR / 32;
  constexpr u32 kCols = KIND == kForward ? TILE / 2 : TILE;  // columns of the results
  // Names of their own, so that the compiler sees that reads of one and copies to another do not
  // meet, and waits for none of them; it tells seven apart.  An operand has two deep tiles, or four.
  constexpr int kP = kTileBytes<TILE, kPByK>, kQ = kTileBytes<TILE, kQByK>;
  constexpr bool kEight = !kPByK && !kQByK;
  __shared__ __attribute__((aligned(128))) char p1[kP], p2[kPByK ? 16 : kP], p3[kPByK ? 16 : kP];
  __shared__ __attribute__((aligned(128))) char q1[kQ], q2[kQByK ? 16 : kQ], q3[kQByK ? 16 : kQ];
  __shared__ __attribute__((aligned(128))) char p0[kEight ? kP + kQ : kP], q0[kEight ? 16 : kQ];
  u32 tr, tc;
  const u32 halves = KIND == kWeight ? 2 : 1;
  const u32 split = KIND == kForward ? 0 : blockIdx.x / (down * halves * across);
  tile_of(KIND == kForward ? blockIdx.x : blockIdx.x % (down * halves * across), down * halves, across, tr, tc);
  const int which = KIND == kWeight && tr >= down;
  const int64_t r0 = (int64_t)(tr - which * down) * TILE, c0 = (int64_t)tc * kCols;
  const u32 wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const u32 wc = wave % WC, wr = wave / WC;

  constexpr int kRP = kRounds<kPByK>, kRQ = kRounds<kQByK>;
  u32 op[kRP], oq[kRQ];
#pragma unroll
  for (int i = 0; i < kRP; ++i)  // in the forward pass gate's columns, then up's
    op[i] = place_of<TILE, kPByK>(KIND == kForward ? i % (kRP / 2) : i, a.ld_p[0], c0, a.cols);
#pragma unroll
  for (int i = 0; i < kRQ; ++i) oq[i] = place_of<TILE, kQByK>(i, a.ld_q[0], r0, a.rows);
  u32 at_p[XB], at_q[YB];
  block_offsets<TILE, kQByK>(at_q, wr * YB * 32);
  if constexpr (KIND == kForward) {  // blocks of gate, then of up
    u32 gate[XB / 2];
    block_offsets<TILE, kPByK>(gate, wc * (XB / 2) * 32);
#pragma unroll
    for (int x = 0; x < XB; ++x) at_p[x] = gate[x % (XB / 2)] + x / (XB / 2) * (TILE / 2) * 128;
  } else {
    block_offsets<TILE, kPByK>(at_p, wc * XB * 32);
  }
  f32x16 acc[XB][YB] = {};
  struct Fragments {
    i16x8 p[kStep / 16][XB], q[kStep / 16][YB];
  };
  // a split has a run of the 64s of k, in the input gradient of gate's and then up's
  constexpr u32 kParts = KIND == kInput ? 2 : 1;
  const u32 units = (u32)((a.k + 63) / 64);
  const u32 from = (u32)((u64)units * kParts * split / splits), to = (u32)((u64)units * kParts * (split + 1) / splits);
  for (u32 part = 0; part < kParts; ++part) {
    const u32 lo = max(from, part * units) - part * units, hi = min(to, (part + 1) * units) - part * units;
    if (KIND != kForward && (from >= (part + 1) * units || to <= part * units)) continue;
    const int64_t k_lo = KIND == kForward ? 0 : (int64_t)lo * 64;
    const int k = (int)((KIND == kForward ? a.k : min(a.k, (int64_t)hi * 64)) - k_lo);
    const u32 steps = (u32)(k + kStep - 1) / kStep, whole = (u32)k / kStep;
    const u32 iq = KIND == kWeight ? which : part, ip = KIND == kInput ? part : 0;
    // where the next copies begin, how far a copy goes, and what is left of k there
    const char* next_q = a.q[iq] + (kQByK ? r0 * a.ld_q[0] + k_lo * 2 : k_lo * a.ld_q[0] + r0 * 2);
    const char* next_p[2] = {a.p[ip] + (kPByK ? c0 * a.ld_p[0] + k_lo * 2 : k_lo * a.ld_p[0] + c0 * 2),
                             KIND == kForward ? a.p[1] + c0 * a.ld_p[0] : nullptr};
    const int64_t far_q = kDeep<kQByK> * (kQByK ? 2 : a.ld_q[0]), far_p = kDeep<kPByK> * (kPByK ? 2 : a.ld_p[0]);
    int left_p = k, left_q = k;
    auto copy_p = [&](char* to, auto all_whole) {
      auto start = [&](auto is_part) {
#pragma unroll
        for (int i = 0; i < kRP; ++i)
          copy_place<TILE, kPByK, decltype(is_part)::value>(to, buffer_at(next_p[KIND == kForward ? i / (kRP / 2) : 0]), op[i], i,
                                                            left_p);
      };
      if (decltype(all_whole)::value || left_p >= kDeep<kPByK>) start(std::false_type{});
      else start(std::true_type{});
      next_p[0] += far_p;
      if constexpr (KIND == kForward) next_p[1] += far_p;
      left_p -= kDeep<kPByK>;
    };
    auto copy_q = [&](char* to, auto all_whole) {
      auto start = [&](auto is_part) {
#pragma unroll
        for (int i = 0; i < kRQ; ++i) copy_place<TILE, kQByK, decltype(is_part)::value>(to, buffer_at(next_q), oq[i], i, left_q);
      };
      if (decltype(all_whole)::value || left_q >= kDeep<kQByK>) start(std::false_type{});
      else start(std::true_type{});
      next_q += far_q;
      left_q -= kDeep<kQByK>;
    };
    // Steps go round J = 0 .. 3.  The tile of step J, or of steps J and J + 1 (J even) where it is deep:
    auto tile_p = [&](auto j) -> char* {
      constexpr int J = decltype(j)::value & 3;
      if constexpr (kPByK) return J < 2 ? p0 : p1;
      else return J == 0 ? p0 : J == 1 ? p1 : J == 2 ? p2 : p3;
    };
    auto tile_q = [&](auto j) -> char* {
      constexpr int J = decltype(j)::value & 3;
      if constexpr (kQByK) return J < 2 ? q0 : q1;
      else return J == 0 ? (kEight ? p0 + kP : q0) : J == 1 ? q1 : J == 2 ? q2 : q3;
    };
    auto read = [&](auto j, Fragments& f) {
      constexpr u32 J = decltype(j)::value & 3;
#pragma unroll
      for (u32 s = 0; s < kStep / 16; ++s) {
#pragma unroll
        for (int y = 0; y < YB; ++y)
          f.q[s][y] = fragment<TILE, kQByK>(tile_q(j), at_q[y], s + (kQByK ? J % 2 * 2 : 0));
#pragma unroll
        for (int x = 0; x < XB; ++x)
          f.p[s][x] = fragment<TILE, kPByK>(tile_p(j), at_p[x], s + (kPByK ? J % 2 * 2 : 0));
      }
    };
    // A step multiplies fragments that are in registers, while those of the next one are read, and starts
    // the copies that fit into what it was itself read from: a step's tile four steps ahead, or
    // with its second step a deep tile three steps ahead.
    auto copies = [&](auto j, u32 s, auto all_whole) {
      constexpr int J = decltype(j)::value;
      const bool small = decltype(all_whole)::value || s + 4 < steps, deep = decltype(all_whole)::value || s + 3 < steps;
      if constexpr (!kPByK || J % 2 == 1)
        if (kPByK ? deep : small) copy_p(tile_p(j), all_whole);
      if constexpr (!kQByK || J % 2 == 1)
        if (kQByK ? deep : small) copy_q(tile_q(j), all_whole);
    };
    auto multiply_and_read = [&](auto j, const Fragments& f, Fragments& next) {
      constexpr int J = decltype(j)::value;
      read(std::integral_constant<int, J + 1>{}, next);
#pragma unroll
      for (u32 s = 0; s < kStep / 16; ++s)
#pragma unroll
        for (int x = 0; x < XB; ++x)
#pragma unroll
          for (int y = 0; y < YB; ++y) acc[x][y] = mfma32<T>(f.p[s][x], f.q[s][y], acc[x][y]);
      // a few reads behind each matrix instruction, so that neither waits for the other
      constexpr int kReads = kStep / 16 * ((kPByK ? 1 : 2) * XB + (kQByK ? 1 : 2) * YB);
      constexpr int kMfma = kStep / 16 * XB * YB;
      constexpr int kEach = (kReads + kMfma - 3) / (kMfma - 2);
      interleave<kMfma, (!kPByK || J % 2 ? kRP : 0) + (!kQByK || J % 2 ? kRQ : 0), kReads, kEach>();
    };
    constexpr int kSmall = (kPByK ? 0 : kRP) + (kQByK ? 0 : kRQ);  // copies started by an even step
    auto step = [&](auto j, const Fragments& f, Fragments& next) {
      constexpr int J = decltype(j)::value;
      copies(j, 0, std::true_type{});
      multiply_and_read(j, f, next);
      // what the next step reads has arrived: deep tiles started by the step before an even one; tiles of
      // one step started two before
      turn<(kPByK || kQByK) && J % 2 == 0 ? kSmall : 8>();
    };
    auto last_steps = [&](auto j, u32 s, const Fragments& f, Fragments& next) {
      if (s >= steps) return;
      copies(j, s, std::false_type{});
      multiply_and_read(j, f, next);
      turn<0>();
    };
    using J0 = std::integral_constant<int, 0>;
    using J1 = std::integral_constant<int, 1>;
    using J2 = std::integral_constant<int, 2>;
    using J3 = std::integral_constant<int, 3>;
    Fragments f, g;
    copy_p(tile_p(J0{}), std::false_type{});
    copy_q(tile_q(J0{}), std::false_type{});
    if (!kPByK && 1 < steps) copy_p(tile_p(J1{}), std::false_type{});
    if (!kQByK && 1 < steps) copy_q(tile_q(J1{}), std::false_type{});
    if (2 < steps) {
      copy_p(tile_p(J2{}), std::false_type{});
      copy_q(tile_q(J2{}), std::false_type{});
    }
    if (!kPByK && 3 < steps) copy_p(tile_p(J3{}), std::false_type{});
    if (!kQByK && 3 < steps) copy_q(tile_q(J3{}), std::false_type{});
    if (whole >= 4) turn<8>();  // the second four steps' copies may still be under way
    else turn<0>();
    read(J0{}, f);
    turn<8>();
    u32 s = 0;
    for (; s + 8 <= whole; s += 4) {  // copies of whole steps only
      step(J0{}, f, g);
      step(J1{}, g, f);
      step(J2{}, f, g);
      step(J3{}, g, f);
    }
#pragma unroll 1
    for (; s < steps; s += 4) {
      last_steps(J0{}, s, f, g);
      last_steps(J1{}, s + 1, g, f);
      last_steps(J2{}, s + 2, f, g);
      last_steps(J3{}, s + 3, g, f);
    }
  }

  // A block's results lie across the lanes by rows, four columns a lane: stored as they are, each store of
  // a wave would touch 32 rows by 16 bytes.  They go through LDS, where the copies no longer need it, and
  // leave by whole rows of the wave's columns.
  constexpr u32 kOf = kPByK ? 2 : 4, kEach = WC * WR / kOf;
  const u32 slot = wave / kEach;
  char* at_slot = slot == 0 ? p0 : p1;
  if constexpr (!kPByK) at_slot = slot == 2 ? p2 : slot == 3 ? p3 : at_slot;
  char* const mine = at_slot + wave % kEach * kStageBytes;
#pragma unroll
  for (int y = 0; y < YB; ++y) {
    const int64_t r = r0 + (wr * YB + y) * 32;
    const ProductLaunch& b = argument<ProductLaunch>();
    if constexpr (KIND == kForward) {
      constexpr int XG = XB / 2, kWide = XG * 32;
      const int64_t c = c0 + wc * kWide;
#pragma unroll
      for (int x = 0; x < XG; ++x)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = gated_value(b.act, acc[x][y][4 * j + e], acc[x + XG][y][4 * j + e]);
          stage_bits<T, kWide>(mine, x * 32 + 8 * j, v);
        }
      flush_bits<T, kWide>(mine, b.out[0], b.ld_out[0], r, b.rows, c, b.cols);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const ProductLaunch& b = argument<ProductLaunch>();
        if (b.kept[0]) {
#pragma unroll
          for (int x = 0; x < XG; ++x)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float v[4] = {acc[x + i * XG][y][4 * j], acc[x + i * XG][y][4 * j + 1], acc[x + i * XG][y][4 * j + 2],
                                  acc[x + i * XG][y][4 * j + 3]};
              stage_bits<T, kWide>(mine, x * 32 + 8 * j, v);
            }
          flush_bits<T, kWide>(mine, b.kept[i], b.ld_kept[i], r, b.rows, c, b.cols);
        }
        if (b.held[0].codes) {
#pragma unroll
          for (int x = 0; x < XG; ++x) hold_block<kWide>(mine, b.held[i], acc[x + i * XG][y], r, b.rows, c + 32 * x, 32 * x, b.cols);
          flush_codes<kWide>(mine, b.held[i], r, b.rows, c, b.cols);
        }
      }
    } else if (splits > 1) {  // fp32, for join_kernel
      const int64_t at = ((int64_t)(split * halves + which) * b.rows + r) * b.cols;
#pragma unroll
      for (int x = 0; x < XB; ++x) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          stage_floats(mine, 8 * j, f32x4{acc[x][y][4 * j], acc[x][y][4 * j + 1], acc[x][y][4 * j + 2], acc[x][y][4 * j + 3]});
        flush_partial(mine, b.ws + at, r, b.rows, c0 + (wc * XB + x) * 32, b.cols);
      }
    } else if (KIND == kInput || (b.out_type != ZERO_F32 && !b.accumulate)) {  // rounded once, to 16 bits
      constexpr int kWide = 64;
      auto store = [&](auto type) {
        using O = decltype(type);
#pragma unroll
        for (int x = 0; x < XB; x += 2) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float v[4] = {acc[x + i][y][4 * j], acc[x + i][y][4 * j + 1], acc[x + i][y][4 * j + 2], acc[x + i][y][4 * j + 3]};
              stage_bits<O, kWide>(mine, i * 32 + 8 * j, v);
            }
          flush_bits<O, kWide>(mine, b.out[which], b.ld_out[which], r, b.rows, c0 + (wc * XB + x) * 32, b.cols);
        }
      };
      if constexpr (KIND == kInput) store(T{});
      else if (b.out_type == ZERO_BF16) store(BF16{});
      else store(F16{});
    } else {
#pragma unroll
      for (int x = 0; x < XB; ++x) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          stage_floats(mine, 8 * j, f32x4{acc[x][y][4 * j], acc[x][y][4 * j + 1], acc[x][y][4 * j + 2], acc[x][y][4 * j + 3]});
        flush_floats(mine, b, which, r, c0 + (wc * XB + x) * 32);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// a few tokens
// ---------------------------------------------------------------------------

// Every weight is read once, and what counts is the bytes in flight and that all CUs have a like share
// of them.  A workgroup has COLS columns of gate and of up, 16 or 32 (a block, where they are held in 8 bits); its waves take turns of 64 of k and work alone: each copies its
// turns' weights and tokens into LDS, whole lines, RING turns ahead, and waits for no other wave before its
// sums are added to theirs.  Weights loaded straight into the registers that the matrix
// instructions take them from, 16 bytes of every row a lane, reached half of the bandwidth: each
// lane of such a load is a line of its own to the L1.  TOKENS: a multiple of 16.
template <class T>
__device__ __forceinline__ f32x4 mfma16(i16x8 p, i16x8 q, f32x4 acc) {
  if constexpr (std::is_same<T, BF16>::value)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, p), __builtin_bit_cast(bf16x8, q), acc, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, p), __builtin_bit_cast(f16x8, q), acc, 0, 0, 0);
}

template <class T, int TOKENS, int COLS, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void few_kernel(const ProductLaunch a) {
  constexpr int N = TOKENS / 16, H = COLS / 16, kRing = N <= 2 ? 3 : 2;
  constexpr int kTurnBytes = (2 * COLS + TOKENS) * 128;  // rows of gate, of up, of tokens
  constexpr int kCopies = kTurnBytes / 1024;
  __shared__ __attribute__((aligned(128))) char s0[WAVES * kTurnBytes], s1[WAVES * kTurnBytes],
      s2[kRing > 2 ? WAVES * kTurnBytes : 16];
  const u32 lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int64_t c0 = (int64_t)blockIdx.x * COLS;
  // Chunk i of 8 rows: lane l fetches the unit of row 8 i + l / 8 whose place is l % 8 (unit j of row r at
  // j ^ (r / 2 % 8)).  Rows beyond the last stand for it.
  u32 off[COLS / 8], off_x[2 * N];
#pragma unroll
  for (u32 i = 0; i < COLS / 8; ++i)
    off[i] = (u32)min((int64_t)(8 * i + lane / 8), a.cols - 1 - c0) * (u32)a.ld_p[0] + ((lane % 8) ^ ((4 * i + lane / 16) % 8)) * 16;
#pragma unroll
  for (u32 i = 0; i < 2 * N; ++i)
    off_x[i] = (u32)min((int64_t)(8 * i + lane / 8), a.rows - 1) * (u32)a.ld_q[0] + ((lane % 8) ^ ((4 * i + lane / 16) % 8)) * 16;
  u32 at = wave * kTurnBytes + lane % 16 * 128 + ((lane / 16) ^ (lane / 2 % 8)) * 16;  // 16 rows further: + 2048
  asm("" : "+v"(at));

  auto copy = [&](char* slot, int64_t u) {
    const int64_t left = a.k - u * 64;
    auto start = [&](auto is_part) {
      auto one = [&](__amdgpu_buffer_rsrc_t from, u32 from_off, u32 i, u32 chunk) {
        char* const to = slot + wave * kTurnBytes + chunk * 1024;
        if (!decltype(is_part)::value || (int64_t)(((lane % 8) ^ ((4 * i + lane / 16) % 8)) * 8) < left)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void*)to, 16, from_off, 0, 0, 0);
        else
          *reinterpret_cast<vec4*>(to + lane * 16) = vec4{0, 0, 0, 0};  // beyond the end of k
      };
#pragma unroll
      for (u32 m = 0; m < 2; ++m)
#pragma unroll
        for (u32 i = 0; i < COLS / 8; ++i) one(buffer_at(a.p[m] + c0 * a.ld_p[0] + u * 128), off[i], i, COLS / 8 * m + i);
#pragma unroll
      for (u32 i = 0; i < 2 * N; ++i) one(buffer_at(a.q[0] + u * 128), off_x[i], i, COLS / 4 + i);
    };
    if (left >= 64) start(std::false_type{});
    else start(std::true_type{});
  };
  f32x4 acc[2][H][N] = {};
  // this wave's turns are 64 of k from 64 (wave + WAVES i) on
  const int64_t all = (a.k + 63) / 64, turns = (all - wave + WAVES - 1) / WAVES;
  const int64_t whole = (a.k / 64 - wave + WAVES - 1) / WAVES;  // of them without an end of k inside
  auto turn = [&](char* slot, int64_t i) {
    if (i >= turns) return;
    // the ring's other turns may be under way still; one with an end of k inside starts fewer copies
    if (i + kRing - 1 < whole) __builtin_amdgcn_s_waitcnt(0x70 | ((kRing - 1) * kCopies & 15) | ((kRing - 1) * kCopies >> 4) << 14);
    else __builtin_amdgcn_s_waitcnt(0x70);
    i16x8 w[2][H][2], x[N][2];
#pragma unroll
    for (u32 s = 0; s < 2; ++s) {
#pragma unroll
      for (u32 m = 0; m < 2; ++m)
#pragma unroll
        for (u32 h = 0; h < H; ++h) w[m][h][s] = *reinterpret_cast<const i16x8*>(slot + ((at ^ (s * 64)) + (H * m + h) * 2048));
#pragma unroll
      for (int t = 0; t < N; ++t) x[t][s] = *reinterpret_cast<const i16x8*>(slot + ((at ^ (s * 64)) + (2 * H + t) * 2048));
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): what was read may be written over
    asm volatile("" ::: "memory");
    if (i + kRing < turns) copy(slot, wave + WAVES * (i + kRing));
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int t = 0; t < N; ++t)
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int h = 0; h < H; ++h) acc[m][h][t] = mfma16<T>(w[m][h][s], x[t][s], acc[m][h][t]);
  };
  if (0 < turns) copy(s0, wave);
  if (1 < turns) copy(s1, wave + WAVES);
  if (kRing > 2 && 2 < turns) copy(s2, wave + 2 * WAVES);
#pragma unroll 1
  for (int64_t i = 0; i < turns; i += kRing) {
    turn(s0, i);
    turn(s1, i + 1);
    if constexpr (kRing > 2) turn(s2, i + 2);
  }

  // sums [wave][gate or up][token][column]
  static_assert(2 * TOKENS * COLS * 4 <= kTurnBytes, "the sums fit where the copies were");
  float* const sums = reinterpret_cast<float*>(s0);
  __syncthreads();
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int t = 0; t < N; ++t)
#pragma unroll
      for (int h = 0; h < H; ++h)
        *reinterpret_cast<f32x4*>(sums + ((wave * 2 + m) * TOKENS + 16 * t + lane % 16) * COLS + 16 * h + lane / 16 * 4) = acc[m][h][t];
  __syncthreads();
  // four columns a thread
#pragma unroll 1
  for (u32 e = threadIdx.x; e < TOKENS * (COLS / 4); e += WAVES * 64) {
    const u32 t = e / (COLS / 4), col = e % (COLS / 4) * 4;
    const int64_t c = c0 + col;
    const u32 n = c < a.cols ? (u32)min(a.cols - c, (int64_t)4) : 0;
    float v[2][4];
#pragma unroll
    for (u32 m = 0; m < 2; ++m) {
      f32x4 f = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (u32 k = 0; k < WAVES; ++k) f += *reinterpret_cast<const f32x4*>(sums + ((k * 2 + m) * TOKENS + t) * COLS + col);
#pragma unroll
      for (u32 j = 0; j < 4; ++j) v[m][j] = j < n ? f[j] : 0.0f;
    }
    if (COLS == kBlock && a.held[0].codes) {
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        u32 top = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) top = max(top, finite_magnitude(v[m][j]));
#pragma unroll
        for (int d = 1; d < 8; d *= 2) top = max(top, (u32)__shfl_xor((int)top, d, 64));
        if (t >= a.rows || n == 0) continue;
        const u32 scale = scale_of(top);
        store_codes4(a.held[m], t, c, v[m], scale, n);
        if (col == 0) a.held[m].scales[t * a.held[m].ld_scales + c / kBlock] = (char)scale;
      }
    }
    if (t < a.rows && n > 0) finish_gated4<T>(a, t, c, v[0], v[1], n);
  }
}

template <class T, int TOKENS>
int few_as(const ProductLaunch& a, hipStream_t s) {
  auto go = [&](auto columns, auto waves) {
    constexpr int C = decltype(columns)::value, W = decltype(waves)::value;
    hipLaunchKernelGGL((few_kernel<T, TOKENS, C, W>), dim3((u32)((a.cols + C - 1) / C)), dim3(W * 64), 0, s, a);
  };
  using Two = std::integral_constant<int, 2>;
  using Four = std::integral_constant<int, 4>;
  const bool many = a.cols > 16 * 512;  // more than two workgroups a CU
  // With 64 tokens their rows are more than the weights' of 16 columns (64 tokens, 4096 x 14336
  // 58 us with 32 columns, 69 with 16; 16 tokens 48 and 47, 4096 x 11008 45 and 37.5).
  if (TOKENS == 64 || a.held[0].codes) {
    a.cols > 32 * 256 ? go(std::integral_constant<int, 32>{}, Two{}) : go(std::integral_constant<int, 32>{}, Four{});
  } else if constexpr (TOKENS < 64) {
    many ? go(std::integral_constant<int, 16>{}, Two{}) : go(std::integral_constant<int, 16>{}, Four{});
  }
  return launched("gated projections");
}

// Whether the copies of 16 bytes find whole units: addresses, strides, and the lengths
// along which an operand's rows lie.  Offsets within a tile are 32 bits.
bool tiles_fit(Product kind, const ProductLaunch& a) {
  auto ok = [](const char* p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 16 == 0 && ld < (1 << 22); };
  const int nq = kind == kForward ? 1 : 2, np = kind == kWeight ? 1 : 2;
  for (int i = 0; i < nq; ++i)
    if (!ok(a.q[i], a.ld_q[i])) return false;
  for (int i = 0; i < np; ++i)
    if (!ok(a.p[i], a.ld_p[i])) return false;
  const bool q_by_k = kind != kWeight, p_by_k = kind == kForward;
  if (a.k < 1 || a.ld_p[0] != a.ld_p[np - 1] || a.ld_q[0] != a.ld_q[nq - 1]) return false;
  return (q_by_k ? a.k : a.rows) % 8 == 0 && (p_by_k ? a.k : a.cols) % 8 == 0;
}

// Adds the splits' sums, four columns a thread, in their order.
template <class T, Product KIND>
__global__ __launch_bounds__(256) void join_kernel(const ProductLaunch a, u32 splits) {
  const int64_t each = a.rows * a.cols, all = each * (KIND == kWeight ? 2 : 1);
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < all; i += (int64_t)gridDim.x * 1024) {
    const int which = i >= each;
    const int64_t r = (i - which * each) / a.cols, c = (i - which * each) % a.cols;
    f32x4 sum = *reinterpret_cast<const f32x4*>(a.ws + i);
#pragma unroll 4
    for (u32 s = 1; s < splits; ++s) sum += *reinterpret_cast<const f32x4*>(a.ws + s * all + i);
    const float v[4] = {sum[0], sum[1], sum[2], sum[3]};
    finish4<T, KIND>(a, which, r, c, v, 4);
  }
}

// The size of the tiles and the number of splits of k.  Few tiles leave CUs without work; splits of a long k
// give it to them, at the price of fp32 partial results that are written and read once more.  The
// estimate is of microseconds, from these measurements: 64 of k take a tile of 256 1.5, of
// 128 0.4 alone on a CU and 0.95 where two share it (the 8192 x 4096 x 14336 forward pass 1498 us with
// tiles of 256, 1873 with 128); a tile begins and ends in 8 and 5; partial results move at 5 TB/s,
// and another launch takes 3.
struct TilePlan {
  int tile;
  u32 splits;
};
constexpr u32 kMaxSplits = 16;
constexpr int64_t kMaxPartialBytes = int64_t(64) << 20;

TilePlan tile_plan(Product kind, const ProductLaunch& a) {
  const int64_t halves = kind == kWeight ? 2 : 1, units = (a.k + 63) / 64 * (kind == kInput ? 2 : 1);
  const int64_t bytes = halves * a.rows * a.cols * 4;
  TilePlan best{128, 1};
  double least = 1e300;
  for (int tile : {128, 256}) {
    const int64_t cols = kind == kForward ? tile / 2 : tile;
    const int64_t tiles = (a.rows + tile - 1) / tile * ((a.cols + cols - 1) / cols) * halves;
    for (u32 n = 1; n <= kMaxSplits; ++n) {
      if (n > 1 && (kind == kForward || units / n < 4 || bytes > kMaxPartialBytes / n || a.cols % 8 != 0)) break;
      const int64_t groups = tiles * n;
      double each, begin, rounds;
      if (tile == 256) each = 1.5, begin = 8.0, rounds = (double)((groups + 255) / 256);
      else if (groups <= 256) each = 0.4, begin = 5.0, rounds = 1.0;
      else each = 0.95, begin = 5.0, rounds = (double)((groups + 511) / 512);
      double t = rounds * (each * (double)units / n + begin);
      if (n > 1) t += 3.0 + 2.0 * n * (double)bytes / 5e6;
      if (t < least) {
        least = t;
        best = TilePlan{tile, n};
      }
    }
  }
  return best;
}

template <class T, Product KIND, int TILE>
int tiled_as(const ProductLaunch& a, u32 splits, hipStream_t s) {
  constexpr int cols = KIND == kForward ? TILE / 2 : TILE;
  const u32 down = (u32)((a.rows + TILE - 1) / TILE), across = (u32)((a.cols + cols - 1) / cols);
  hipLaunchKernelGGL((tiled_kernel<T, KIND, TILE>), dim3(down * across * (KIND == kWeight ? 2 : 1) * splits),
                     dim3(kTileThreads<TILE>), 0, s, a, down, across, splits);
  return launched(KIND == kForward ? "gated projections" : KIND == kInput ? "gated input gradient" : "gated weight gradient");
}

template <class T, Product KIND>
int tiled_of(const ProductLaunch& a, hipStream_t s) {
  if constexpr (KIND == kForward) {
    if (a.rows <= 16) return few_as<T, 16>(a, s);
    if (a.rows <= 32) return few_as<T, 32>(a, s);
    if (a.rows <= 64) return few_as<T, 64>(a, s);
  }
  const TilePlan plan = tile_plan(KIND, a);
  if (int rc = plan.tile == 256 ? tiled_as<T, KIND, 256>(a, plan.splits, s) : tiled_as<T, KIND, 128>(a, plan.splits, s)) return rc;
  if constexpr (KIND != kForward) {
    if (plan.splits > 1) {
      const int64_t all = a.rows * a.cols * (KIND == kWeight ? 2 : 1);
      hipLaunchKernelGGL((join_kernel<T, KIND>), dim3((u32)std::min<int64_t>((all + 1023) / 1024, 4096)), dim3(256), 0, s, a,
                         plan.splits);
      return launched("gated products (join)");
    }
  }
  return ZERO_OK;
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
  if (t != ZERO_F32 && tiles_fit(KIND, a)) return t == ZERO_BF16 ? tiled_of<BF16, KIND>(a, s) : tiled_of<F16, KIND>(a, s);
  switch (t) {
    case ZERO_F32: return product_as<F32, KIND>(a, s);
    case ZERO_BF16: return product_as<BF16, KIND>(a, s);
    default: return product_as<F16, KIND>(a, s);
  }
}

}  // namespace

int64_t product_ws_bytes(int64_t tokens, int64_t dim, int64_t hidden) {
  const double most = 4.0 * kMaxSplits * (double)dim * (double)std::max(tokens, 2 * hidden);
  return most < (double)kMaxPartialBytes ? (int64_t)most : kMaxPartialBytes;
}

int launch_product(Product kind, const ProductLaunch& a, zero_dtype_t t, void* stream) {
  switch (kind) {
    case kForward: return product_of<kForward>(a, t, (hipStream_t)stream);
    case kInput: return product_of<kInput>(a, t, (hipStream_t)stream);
    default: return product_of<kWeight>(a, t, (hipStream_t)stream);
  }
}

}  // namespace zk
