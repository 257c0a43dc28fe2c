// What the gated block's matrix products share: the layout of an operand's tile in LDS and
// how matrix instructions read it, the order of tiles, and what becomes of the results.
#ifndef ZERO_PRODUCTS_H_
#define ZERO_PRODUCTS_H_

#include "held.h"

namespace zk {

// Products of any type, size, stride and alignment.
int launch_product_any(Product kind, const ProductLaunch& a, zero_dtype_t t, void* stream);
// Adds the sums of splits in their order and finishes them.
int launch_join(Product kind, const ProductLaunch& a, zero_dtype_t t, uint32_t splits, void* stream);

namespace {

constexpr u32 kMaxSplits = 32;  // of fp32 sums; 16 of 16-bit products, whose steps are short beside a partial result
constexpr int64_t kMaxPartialBytes = int64_t(64) << 20;

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef short i16x8 __attribute__((ext_vector_type(8)));
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

template <class T>
__device__ __forceinline__ float gated_value(int32_t act, float g, float u) {
  return g * (act == kSilu ? gate_of<T, kSilu>(g).p : gate_of<T, kGelu>(g).p) * u;
}

// The same of the forward pass: gate and up.
template <class T>
__device__ __forceinline__ void finish_gated4(const ProductLaunch& a, int64_t r, int64_t c, const float g[4], const float u[4],
                                              u32 n) {
  float v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = gated_value<T>(a.act, g[j], u[j]);
  store4<T>(a.out[0] + r * a.ld_out[0] + c * T::bytes, v, n);
  if (a.kept[0]) {
    store4<T>(a.kept[0] + r * a.ld_kept[0] + c * T::bytes, g, n);
    store4<T>(a.kept[1] + r * a.ld_kept[1] + c * T::bytes, u, n);
  }
}

// ---------------------------------------------------------------------------
// an operand's tile
// ---------------------------------------------------------------------------

// LDS holds an operand as its rows lie in memory.  Rows of k are 64 of k long, 128 bytes:
// unit (16 bytes) j of row i sits at j ^ (i / 2 % 8), so that the 16-byte reads of 16 lanes in
// neighbouring rows meet every bank once.  Rows of the other index ([32 k][TILE]) are read
// transposed, 4 rows of 16 columns by 16 lanes: unit j of row k sits at j ^ 2 (k % 4) in
// tiles of 128; in tiles of 256, whose kernels have no registers for the addresses that this
// takes, at j ^ 2 (k % 2), with 64 bytes left out before every odd pair of rows.  Either way
// the 4 rows that 16 lanes read lie in different banks; what the other lanes of a wave read at the same time is not
// kept apart from them, and the kernels that read transposed count 1.4 to 2.0 conflict cycles an LDS
// instruction (the forward pass, whose rows are of k, 0.2).
constexpr int kStep = 32;
template <bool DEEP>
constexpr int kDeep = DEEP ? 2 * kStep : kStep;  // of k, copied at a time
template <bool DEEP>
constexpr int kRounds = DEEP ? 4 : 2;            // 16 bytes a thread and round

// Where the 1024 bytes of chunk c of a tile begin.
template <int TILE, bool BY_K>
__device__ __forceinline__ u32 chunk_at(u32 c) {
  return c * 1024 + (TILE == 256 && !BY_K ? (c + 1) / 2 * 64 : 0);
}
template <int TILE>
__device__ __forceinline__ u32 swizzle(u32 k) {
  return TILE == 256 ? k % 2 * 2 : k % 4 * 2;
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
template <class T>
__device__ __forceinline__ f32x4 mfma16(i16x8 p, i16x8 q, f32x4 acc) {
  if constexpr (std::is_same<T, BF16>::value)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, p), __builtin_bit_cast(bf16x8, q), acc, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, p), __builtin_bit_cast(f16x8, q), acc, 0, 0, 0);
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

// ---------------------------------------------------------------------------
// results by way of LDS
// ---------------------------------------------------------------------------

// A block's results lie across the lanes by rows, four columns a lane: stored as they are, each store of
// a wave would touch 32 rows by 16 bytes.  They go through LDS and leave by whole rows of the wave's
// columns.  32 rows of a wave, each of WIDE 16-bit results, 32 fp32 ones or WIDE codes, 16 bytes apart from the next
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
// To `which` result, the weight gradient's added to what is there where asked.
template <class T, Product KIND>
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
    finish4<T, KIND>(a, which, r + row, col, v, (u32)min(a.cols - col, (int64_t)4));
  }
  __builtin_amdgcn_wave_barrier();
}

// fp32 results, `out` at row 0 and column 0
__device__ __forceinline__ void flush_f32(const char* s, char* out, int64_t ld, int64_t r, int64_t rows, int64_t c, int64_t cols) {
  const u32 lane = threadIdx.x & 63;
  const int64_t col = c + lane % 8 * 4;
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (u32 i = 0; i < 32; i += 8) {
    const u32 row = i + lane / 8;
    const f32x4 q = *reinterpret_cast<const f32x4*>(s + row * 144 + lane % 8 * 16);
    if (r + row >= rows || col >= cols) continue;
    const float v[4] = {q[0], q[1], q[2], q[3]};
    store4<F32>(out + (r + row) * ld + col * 4, v, (u32)min(cols - col, (int64_t)4));
  }
  __builtin_amdgcn_wave_barrier();
}

// A split's sums have rows of whole 16 bytes.
__host__ __device__ __forceinline__ int64_t partial_cols(int64_t cols) { return (cols + 3) & ~int64_t(3); }
// `out` at row r, rows of partial_cols() columns
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

template <class T, int WIDE>
__device__ __forceinline__ void flush_as(const char* s, char* out, int64_t ld, int64_t r, int64_t rows, int64_t c, int64_t cols) {
  if constexpr (T::bytes == 4) flush_f32(s, out, ld, r, rows, c, cols);
  else flush_bits<T, WIDE>(s, out, ld, r, rows, c, cols);
}

// What a wave's blocks of 32 x 32 results become, rows from r0 on and columns from c0 on; in the forward pass
// half of the blocks are of gate, then of up.  mine: kStageBytes of LDS.
template <class T, Product KIND, int XB, int YB>
__device__ __forceinline__ void finish_tile(const f32x16 (&acc)[XB][YB], char* mine, int64_t r0, int64_t c0, int which, u32 split,
                                            u32 splits) {
#pragma unroll
  for (int y = 0; y < YB; ++y) {
    const int64_t r = r0 + y * 32;
    const ProductLaunch& b = argument<ProductLaunch>();
    if constexpr (KIND == kForward) {
      constexpr int XG = XB / 2, kWide = XG * 32;
      static_assert(T::bytes == 2 || XG == 1, "fp32 results are staged 32 columns at a time");
#pragma unroll
      for (int x = 0; x < XG; ++x)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = gated_value<T>(b.act, acc[x][y][4 * j + e], acc[x + XG][y][4 * j + e]);
          if constexpr (T::bytes == 4) stage_floats(mine, 8 * j, f32x4{v[0], v[1], v[2], v[3]});
          else stage_bits<T, kWide>(mine, x * 32 + 8 * j, v);
        }
      flush_as<T, kWide>(mine, b.out[0], b.ld_out[0], r, b.rows, c0, b.cols);
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
              if constexpr (T::bytes == 4) stage_floats(mine, 8 * j, f32x4{v[0], v[1], v[2], v[3]});
              else stage_bits<T, kWide>(mine, x * 32 + 8 * j, v);
            }
          flush_as<T, kWide>(mine, b.kept[i], b.ld_kept[i], r, b.rows, c0, b.cols);
        }
        if (b.held[0].codes) {
#pragma unroll
          for (int x = 0; x < XG; ++x) hold_block<kWide>(mine, b.held[i], acc[x + i * XG][y], r, b.rows, c0 + 32 * x, 32 * x, b.cols);
          flush_codes<kWide>(mine, b.held[i], r, b.rows, c0, b.cols);
        }
      }
    } else if (splits > 1) {  // fp32, for join_kernel
      const int64_t wide = partial_cols(b.cols), at = ((int64_t)(split * (KIND == kWeight ? 2 : 1) + which) * b.rows + r) * wide;
#pragma unroll
      for (int x = 0; x < XB; ++x) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          stage_floats(mine, 8 * j, f32x4{acc[x][y][4 * j], acc[x][y][4 * j + 1], acc[x][y][4 * j + 2], acc[x][y][4 * j + 3]});
        flush_partial(mine, b.ws + at, r, b.rows, c0 + x * 32, wide);
      }
    } else if ((KIND == kInput && T::bytes == 2) || (KIND == kWeight && b.out_type != ZERO_F32 && !b.accumulate)) {  // rounded once, to 16 bits
      constexpr int kPair = XB < 2 ? 1 : 2, kWide = kPair * 32;
      auto store = [&](auto type) {
        using O = decltype(type);
#pragma unroll
        for (int x = 0; x < XB; x += kPair) {
#pragma unroll
          for (int i = 0; i < kPair; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float v[4] = {acc[x + i][y][4 * j], acc[x + i][y][4 * j + 1], acc[x + i][y][4 * j + 2], acc[x + i][y][4 * j + 3]};
              stage_bits<O, kWide>(mine, i * 32 + 8 * j, v);
            }
          flush_bits<O, kWide>(mine, b.out[which], b.ld_out[which], r, b.rows, c0 + x * 32, b.cols);
        }
      };
      if constexpr (KIND == kInput && T::bytes == 2) store(T{});
      else if (b.out_type == ZERO_BF16) store(BF16{});
      else store(F16{});
    } else {
#pragma unroll
      for (int x = 0; x < XB; ++x) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          stage_floats(mine, 8 * j, f32x4{acc[x][y][4 * j], acc[x][y][4 * j + 1], acc[x][y][4 * j + 2], acc[x][y][4 * j + 3]});
        flush_floats<T, KIND>(mine, b, which, r, c0 + x * 32);
      }
    }
  }
}

// The waves' sums of gate and up for few tokens, added and finished.  sums: WAVES * 2 * TOKENS * COLS floats of LDS.
template <class T, int TOKENS, int COLS, int WAVES>
__device__ __forceinline__ void finish_few(const f32x4 (&acc)[2][COLS / 16][TOKENS / 16], float* sums, const ProductLaunch& a,
                                           int64_t c0) {
  constexpr int N = TOKENS / 16, H = COLS / 16;
  const u32 lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  // sums [wave][gate or up][token][column]
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

}  // namespace
}  // namespace zk

#endif  // ZERO_PRODUCTS_H_
