// HIP kernels for gfx950 (CDNA4): the gated block's products for fp32, and for 16-bit operands
// whose addresses, strides or lengths are not whole units of 16 bytes; and the joining of
// sums that were split.
#include <algorithm>

#include "products.h"

namespace zk {
namespace {

// A unit is 16 bytes, a step 128 bytes of k: 64 of 16 bits, 32 of 32.
template <class T>
constexpr int kUnit = 16 / T::bytes;
template <class T>
constexpr int kAnyStep = 128 / T::bytes;

// The first n elements at p, zeros behind them.  end: of the tensor.
template <class T>
__device__ __forceinline__ vec4 unit_of(const char* p, const char* end, u32 n) {
  vec4 q = {0, 0, 0, 0};
  if (n == 0) return q;
  if (end - p >= 16) {
    q = *reinterpret_cast<const vec4_any*>(p);
    asm volatile("" : "+v"(n));
#pragma unroll
    for (u32 i = 0; i < 4; ++i) {
      if constexpr (T::bytes == 4) q[i] = i < n ? q[i] : 0;
      else q[i] = 2 * i + 1 < n ? q[i] : 2 * i < n ? q[i] & 0xffffu : 0;
    }
  } else {
#pragma unroll 1
    for (u32 j = 0; j < n; ++j) {
      u32 e;
      if constexpr (T::bytes == 4) e = reinterpret_cast<const u32*>(p)[j];
      else e = (u32)reinterpret_cast<const uint16_t*>(p)[j] << (16 * (j % 2));
#pragma unroll
      for (u32 i = 0; i < 4; ++i) q[i] |= i == j * T::bytes / 4 ? e : 0;
    }
  }
  return q;
}

// ---------------------------------------------------------------------------
// tiles
// ---------------------------------------------------------------------------

// Tiles of SIDE x SIDE results, 128 (of gate and up in the forward pass 128 x 64 each) or 64, four waves of a quarter
// each.  The operands go through registers, which takes any address, two steps before they
// are multiplied, into one of two tiles in LDS; a step has one barrier.  fp32 tiles lie as 16-bit
// ones do where their rows are of k: a matrix instruction's k are one element of every unit that the
// lanes read.  4096 tokens of bf16, 2049 x 5503: forward 283 us, input gradient 410, weight
// gradient 292 (653, 451 and 633 TFLOP/s; two tiles share a CU, and its L1 takes two lines for every 128
// bytes that begin inside one); tiles of 64 x 64, loaded one step ahead under masks, took 640, 1118
// and 1510.  1024 tokens of fp32, 2048 x 5504: 392, 358 and 402 us, of a floor of 295 at the rate of fp32
// matrix instructions.  Rows of the other index, [32 k][SIDE] fp32, are read element by element; every
// second four of them have their halves of 64 columns in turn exchanged by 32, so that the two halves
// of a wave meet different banks.
template <int SIDE>
constexpr int kOperand = SIDE * 128;  // bytes

template <class T, bool BY_K, int SIDE>
constexpr u32 kLanes = BY_K ? 8 : SIDE / kUnit<T>;      // of a row
template <class T, bool BY_K, int SIDE>
constexpr u32 kRowsEach = 256 / kLanes<T, BY_K, SIDE>;  // rows of a round; SIDE / 32 rounds are a tile

// This thread's place in LDS of the first round; each round is 4096 bytes further.
template <class T, bool BY_K, int SIDE>
__device__ __forceinline__ u32 put_at() {
  const u32 t = threadIdx.x, row = t / kLanes<T, BY_K, SIDE>, unit = t % kLanes<T, BY_K, SIDE>;
  if constexpr (BY_K) return row * 128 + (unit ^ (row / 2 % 8)) * 16;
  else if constexpr (T::bytes == 2) return row * (SIDE * 2) + (unit ^ swizzle<SIDE>(row)) * 16;
  else return row * (SIDE * 4) + (unit ^ (row / 4 % 2 * 8)) * 16;
}

// Whole steps are loaded with neither branches nor masks: rows (columns) beyond the matrix's ni are replaced by others
// of it, and units that begin in a row of columns may read on into the next row; what comes of either is
// not stored.  The byte offset of this thread's unit of round q of a tile that begins at i0:
template <class T, bool BY_K, int SIDE>
__device__ __forceinline__ int64_t offset_of(int q, int64_t ld, int64_t i0, int64_t ni) {
  const u32 t = threadIdx.x, row = q * kRowsEach<T, BY_K, SIDE> + t / kLanes<T, BY_K, SIDE>, unit = t % kLanes<T, BY_K, SIDE>;
  if constexpr (BY_K) return min((int64_t)row, ni - 1 - i0) * ld + unit * 16;
  else return (int64_t)row * ld + (i0 + unit * kUnit<T> < ni ? unit * 16 : 0);
}
// The number of such steps: the last row of columns is not among them.
template <class T, bool BY_K>
__device__ __forceinline__ int64_t whole_steps(int64_t ni, int64_t nk) {
  return BY_K ? nk / kAnyStep<T> : ni >= kUnit<T> ? (nk - 1) / kAnyStep<T> : 0;
}

// This thread's unit of round q of any step: from k0 on, of a matrix at p with ni rows (columns) and nk of k.
template <class T, bool BY_K, int SIDE>
__device__ __forceinline__ vec4 edge_unit(int q, const char* p, const char* end, int64_t ld, int64_t i0, int64_t ni, int64_t k0,
                                          int64_t nk) {
  const u32 t = threadIdx.x, row = q * kRowsEach<T, BY_K, SIDE> + t / kLanes<T, BY_K, SIDE>, unit = t % kLanes<T, BY_K, SIDE> * kUnit<T>;
  const int64_t i = i0 + (BY_K ? row : unit), k = k0 + (BY_K ? unit : row), left = BY_K ? nk - k : ni - i;
  const int64_t at = BY_K ? i * ld + k * T::bytes : k * ld + i * T::bytes;
  return unit_of<T>(p + at, end, i < ni && k < nk ? (u32)min(left, (int64_t)kUnit<T>) : 0);
}

// This lane's offset of the block of 32 rows (columns) from i0 on.
template <class T, bool BY_K, int SIDE>
__device__ __forceinline__ u32 any_offset(u32 i0) {
  const u32 lane = threadIdx.x & 63;
  if constexpr (BY_K || T::bytes == 2) {
    u32 at[1];
    block_offsets<SIDE, BY_K>(at, i0);
    return at[0];
  } else {
    return lane / 32 * (SIDE * 16) + ((i0 + lane % 32) ^ (lane / 32 * 32)) * 4;
  }
}

// Part s of a step's four: lane l has row (column) l % 32 and a unit of k.
template <class T, bool BY_K, int SIDE>
__device__ __forceinline__ vec4 any_fragment(const char* lds, u32 at, u32 s) {
  if constexpr (BY_K) {
    return __builtin_bit_cast(vec4, fragment<SIDE, true>(lds, at, s));
  } else if constexpr (T::bytes == 2) {
    return __builtin_bit_cast(vec4, fragment<SIDE, false>(lds, at, s));
  } else {
    vec4 v;
#pragma unroll
    for (u32 j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const u32*>(lds + at + s * (SIDE * 32) + j * (SIDE * 4));
    return v;
  }
}

template <class T>
__device__ __forceinline__ f32x16 any_mfma32(vec4 p, vec4 q, f32x16 acc) {
  if constexpr (T::bytes == 2) {
    return mfma32<T>(__builtin_bit_cast(i16x8, p), __builtin_bit_cast(i16x8, q), acc);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(p[j]), __uint_as_float(q[j]), acc, 0, 0, 0);
    return acc;
  }
}

template <class T, Product KIND, int SIDE>
__global__ __launch_bounds__(256, SIDE == 128 ? 2 : 4) void any_kernel(const ProductLaunch a, u32 down, u32 across, u32 splits) {
  constexpr bool kQByK = KIND != kWeight, kPByK = KIND == kForward;
  constexpr int B = SIDE / 64, R = SIDE / 32;  // blocks of a wave, rounds of an operand
  static_assert(KIND != kForward || B == 2, "a wave has a block of gate and one of up");
  __shared__ __attribute__((aligned(128))) char s0[2 * kOperand<SIDE>], s1[2 * kOperand<SIDE>];  // P, then Q
  const u32 halves = KIND == kWeight ? 2 : 1;
  const u32 split = KIND == kForward ? 0 : blockIdx.x / (down * halves * across);
  u32 tr, tc;
  tile_of(KIND == kForward ? blockIdx.x : blockIdx.x % (down * halves * across), down * halves, across, tr, tc);
  const int which = KIND == kWeight && tr >= down;
  const int64_t r0 = (int64_t)(tr - which * down) * SIDE, c0 = (int64_t)tc * (KIND == kForward ? SIDE / 2 : SIDE);
  const u32 wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), wc = wave % 2, wr = wave / 2;

  u32 at_p[B], at_q[B];
#pragma unroll
  for (int x = 0; x < B; ++x) {
    at_p[x] = any_offset<T, kPByK, SIDE>(KIND == kForward ? x * 64 + wc * 32 : (wc * B + x) * 32);
    at_q[x] = any_offset<T, kQByK, SIDE>((wr * B + x) * 32);
  }
  f32x16 acc[B][B] = {};
  auto multiply = [&](const char* lds) {
#pragma unroll
    for (u32 s = 0; s < 4; ++s) {
      vec4 p[B], q[B];
#pragma unroll
      for (int x = 0; x < B; ++x) p[x] = any_fragment<T, kPByK, SIDE>(lds, at_p[x], s);
#pragma unroll
      for (int y = 0; y < B; ++y) q[y] = any_fragment<T, kQByK, SIDE>(lds + kOperand<SIDE>, at_q[y], s);
#pragma unroll
      for (int x = 0; x < B; ++x)
#pragma unroll
        for (int y = 0; y < B; ++y) acc[x][y] = any_mfma32<T>(p[x], q[y], acc[x][y]);
    }
  };
  const u32 put_p = put_at<T, kPByK, SIDE>(), put_q = put_at<T, kQByK, SIDE>();
  auto put = [&](char* to, const vec4 (&r)[2 * R]) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      *reinterpret_cast<vec4*>(to + put_p + i * 4096) = r[i];
      *reinterpret_cast<vec4*>(to + kOperand<SIDE> + put_q + i * 4096) = r[R + i];
    }
  };
  // a split has a run of the steps, in the input gradient of gate's and then up's
  constexpr int kParts = KIND == kInput ? 2 : 1;
  const int64_t steps = (a.k + kAnyStep<T> - 1) / kAnyStep<T>;
  const int64_t from = steps * kParts * split / splits, to = steps * kParts * (split + 1) / splits;
#pragma unroll 1
  for (int part = 0; part < kParts; ++part) {
    const ProductLaunch& b = argument<ProductLaunch>();
    const int64_t lo = max(from - part * steps, (int64_t)0), hi = min(to - part * steps, steps);
    const int iq = KIND == kWeight ? which : part, ip = KIND == kInput ? part : 0;
    const char* const q = b.q[iq];
    const char* const p = b.p[ip];
    const int64_t ld_q = b.ld_q[iq], ld_p = b.ld_p[ip];
    const int64_t whole = min(hi, min(whole_steps<T, kPByK>(b.cols, b.k), whole_steps<T, kQByK>(b.rows, b.k)));
    int64_t s = lo;
    if (lo < whole) {
      int64_t op[R], oq[R];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        op[i] = offset_of<T, kPByK, SIDE>(KIND == kForward ? i % 2 : i, KIND == kForward && i >= 2 ? b.ld_p[1] : ld_p, c0, b.cols);
        oq[i] = offset_of<T, kQByK, SIDE>(i, ld_q, r0, b.rows);
      }
      const int64_t far_p = kPByK ? 128 : kAnyStep<T> * ld_p, far_q = kQByK ? 128 : kAnyStep<T> * ld_q;
      const char* next_p = p + (kPByK ? c0 * ld_p : c0 * T::bytes) + lo * far_p;
      const char* next_up = KIND == kForward ? b.p[1] + c0 * b.ld_p[1] + lo * far_p : nullptr;
      const char* next_q = q + (kQByK ? r0 * ld_q : r0 * T::bytes) + lo * far_q;
      auto get = [&](vec4 (&r)[2 * R]) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
          r[i] = *reinterpret_cast<const vec4_any*>((KIND == kForward && i >= 2 ? next_up : next_p) + op[i]);
          r[R + i] = *reinterpret_cast<const vec4_any*>(next_q + oq[i]);
        }
        next_p += far_p;
        next_up += far_p;
        next_q += far_q;
        __builtin_amdgcn_sched_barrier(0);  // the loads first: what follows waits for earlier ones only
      };
      vec4 r[2 * R], n[2 * R];
      get(r);
      if (lo + 1 < whole) get(n);
      put(s0, r);
      __syncthreads();
#pragma unroll 1
      for (; s + 3 < whole; s += 2) {
        get(r);
        multiply(s0);
        put(s1, n);
        __syncthreads();
        get(n);
        multiply(s1);
        put(s0, r);
        __syncthreads();
      }
      // one to three steps are left
      const int64_t left = whole - s;
      if (left > 2) get(r);
      multiply(s0);
      if (left > 1) {
        put(s1, n);
        __syncthreads();
        multiply(s1);
      }
      if (left > 2) {
        put(s0, r);
        __syncthreads();
        multiply(s0);
      }
      s = whole;
      __syncthreads();
    }
#pragma unroll 1
    for (; s < hi; ++s) {
      vec4 r[2 * R];
      const int64_t k0 = s * kAnyStep<T>;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int ip2 = KIND == kForward && i >= 2 ? 1 : ip;
        r[i] = edge_unit<T, kPByK, SIDE>(KIND == kForward ? i % 2 : i, b.p[ip2], b.p_end[ip2], b.ld_p[ip2], c0, b.cols, k0, b.k);
        r[R + i] = edge_unit<T, kQByK, SIDE>(i, q, b.q_end[iq], ld_q, r0, b.rows, k0, b.k);
      }
      put(s0, r);
      __syncthreads();
      multiply(s0);
      __syncthreads();
    }
  }
  static_assert(2 * kStageBytes <= sizeof(s0), "two waves' results fit");
  finish_tile<T, KIND, B, B>(acc, (wave < 2 ? s0 : s1) + wave % 2 * kStageBytes, r0 + wr * B * 32, c0 + wc * (KIND == kForward ? 32 : B * 32), which, split, splits);
}

// ---------------------------------------------------------------------------
// a few tokens
// ---------------------------------------------------------------------------

// As few_kernel does, every weight is read once, by waves that work alone: a turn of 128 bytes of k of all rows
// is in registers two turns ahead, and goes through LDS to the lanes that multiply it.  One token of bf16, 4095 x 11007, with
// weights from HBM: 40 us (4.5 TB/s), 59 with the tiles above; of fp32, 4096 x 11008: 74 (4.9 TB/s) and 279.
template <class T>
__device__ __forceinline__ f32x4 any_mfma16(vec4 p, vec4 q, f32x4 acc) {
  if constexpr (T::bytes == 2) {
    return mfma16<T>(__builtin_bit_cast(i16x8, p), __builtin_bit_cast(i16x8, q), acc);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(p[j]), __uint_as_float(q[j]), acc, 0, 0, 0);
    return acc;
  }
}

template <class T, int TOKENS, int COLS>
__global__ __launch_bounds__(256) void few_any_kernel(const ProductLaunch a) {
  constexpr int WAVES = 4, N = TOKENS / 16, H = COLS / 16, kChunks = (2 * COLS + TOKENS) / 8, kTurnBytes = kChunks * 1024;
  __shared__ __attribute__((aligned(128))) char lds[WAVES * kTurnBytes];
  const u32 lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int64_t c0 = (int64_t)blockIdx.x * COLS;
  char* const mine = lds + wave * kTurnBytes;
  // chunk i of 8 rows: lane l has unit l % 8 of row l / 8
  const u32 row = lane / 8, unit = lane % 8;
  const int64_t off[3] = {row * a.ld_p[0] + unit * 16, row * a.ld_p[1] + unit * 16, row * a.ld_q[0] + unit * 16};
  const int64_t turns = (a.k + kAnyStep<T> - 1) / kAnyStep<T>;
  auto get = [&](int64_t u, vec4 (&r)[kChunks]) {
    if (u >= turns) return;
    const ProductLaunch& b = argument<ProductLaunch>();
    const int64_t k0 = u * kAnyStep<T>, k = k0 + unit * kUnit<T>;
    const bool whole = k0 + kAnyStep<T> <= b.k;
    u32 row_now = row;
    asm volatile("" : "+v"(row_now));  // no lane masks held through the loop
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int m = i / (COLS / 8) < 2 ? i / (COLS / 8) : 2, j = m < 2 ? i % (COLS / 8) : i - COLS / 4;
      const int64_t ld = m < 2 ? b.ld_p[m % 2] : b.ld_q[0], at = (m < 2 ? c0 : 0) + 8 * j;
      const bool there = at + row_now < (m < 2 ? b.cols : b.rows);
      const char* const p = (m < 2 ? b.p[m % 2] : b.q[0]) + at * ld + k0 * T::bytes + off[m];
      if (whole) {
        vec4 v = {0, 0, 0, 0};
        if (there) v = *reinterpret_cast<const vec4_any*>(p);
        r[i] = v;
      } else {
        r[i] = unit_of<T>(p, m < 2 ? b.p_end[m % 2] : b.q_end[0], there && k < b.k ? (u32)min(b.k - k, (int64_t)kUnit<T>) : 0);
      }
    }
  };
  // chunks 2 i and 2 i + 1 hold 16 rows: row r's unit j lies at j ^ (r / 2 % 8)
  u32 put[2];
#pragma unroll
  for (u32 i = 0; i < 2; ++i) put[i] = (8 * i + row) * 128 + (unit ^ ((4 * i + row / 2) % 8)) * 16;
  const u32 at = lane % 16 * 128 + ((lane / 16) ^ (lane / 2 % 8)) * 16;
  f32x4 acc[2][H][N] = {};
  auto turn = [&](int64_t u, vec4 (&r)[kChunks]) {
    if (u >= turns) return;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) *reinterpret_cast<vec4*>(mine + i / 2 * 2048 + put[i % 2]) = r[i];
    __builtin_amdgcn_wave_barrier();
    get(u + 2 * WAVES, r);
#pragma unroll
    for (u32 s = 0; s < 2; ++s) {
      vec4 x[N];
#pragma unroll
      for (int t = 0; t < N; ++t) x[t] = *reinterpret_cast<const vec4*>(mine + (at ^ (s * 64)) + (2 * H + t) * 2048);
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const vec4 w = *reinterpret_cast<const vec4*>(mine + (at ^ (s * 64)) + (H * m + h) * 2048);
#pragma unroll
          for (int t = 0; t < N; ++t) acc[m][h][t] = any_mfma16<T>(w, x[t], acc[m][h][t]);
        }
    }
    __builtin_amdgcn_wave_barrier();
  };
  vec4 r[kChunks], n[kChunks];
  get(wave, r);
  get(wave + WAVES, n);
#pragma unroll 1
  for (int64_t u = wave; u < turns; u += 2 * WAVES) {
    turn(u, r);
    turn(u + WAVES, n);
  }
  static_assert(2 * TOKENS * COLS * 4 <= kTurnBytes, "the sums fit where the turns were");
  finish_few<T, TOKENS, COLS, WAVES>(acc, reinterpret_cast<float*>(lds), argument<ProductLaunch>(), c0);
}

template <class T, int TOKENS>
int few_any_as(const ProductLaunch& a, hipStream_t s) {
  auto go = [&](auto columns) {
    constexpr int C = decltype(columns)::value;
    hipLaunchKernelGGL((few_any_kernel<T, TOKENS, C>), dim3((u32)((a.cols + C - 1) / C)), dim3(256), 0, s, a);
  };
  // 32 columns are a block of 8 bits; 16 give twice the workgroups (64 tokens of bf16, 4095 x 11007 83 us and 90,
  // 2047 x 4001 21 and 29; of fp32 221 and 233, 42 and 66)
  if (a.held[0].codes) go(std::integral_constant<int, 32>{});
  else go(std::integral_constant<int, 16>{});
  return launched("gated projections");
}

// ---------------------------------------------------------------------------
// joining
// ---------------------------------------------------------------------------

// Adds the splits' sums, four columns a thread, in their order.
template <class T, Product KIND>
__global__ __launch_bounds__(256) void join_kernel(const ProductLaunch a, u32 splits) {
  const int64_t wide = partial_cols(a.cols), each = a.rows * wide, all = each * (KIND == kWeight ? 2 : 1);
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < all; i += (int64_t)gridDim.x * 1024) {
    const int which = i >= each;
    const int64_t r = (i - which * each) / wide, c = (i - which * each) % wide;
    f32x4 sum = *reinterpret_cast<const f32x4*>(a.ws + i);
#pragma unroll 4
    for (u32 s = 1; s < splits; ++s) sum += *reinterpret_cast<const f32x4*>(a.ws + s * all + i);
    const float v[4] = {sum[0], sum[1], sum[2], sum[3]};
    finish4<T, KIND>(a, which, r, c, v, (u32)min(a.cols - c, (int64_t)4));
  }
}

template <class T, Product KIND>
int join_as(const ProductLaunch& a, u32 splits, hipStream_t s) {
  const int64_t all = a.rows * partial_cols(a.cols) * (KIND == kWeight ? 2 : 1);
  hipLaunchKernelGGL((join_kernel<T, KIND>), dim3((u32)std::min<int64_t>((all + 1023) / 1024, 4096)), dim3(256), 0, s, a, splits);
  return launched("gated products (join)");
}

// The side of the tiles and the number of splits of k, by an estimate of microseconds: what a step takes a tile alone on its
// CU, or a CU full of them (2 of 128, 4 of 64); partial results move at 5 TB/s, and another launch takes 3.  Both
// products of the backward pass, fp32: 593 tokens, 64 x 5936, 95 us with tiles of 128 alone, 45 with 64, 39 with
// up to 32 splits in place of 16; 151 tokens, 96 x 10912, 123, 59 and 46; bf16, 91 tokens, 512 x 4674, 26, 22 and 26.
// The forward pass has neither: more than 64 tokens are tiles of 128 x 64, few of them where hidden is small, each with
// all of k (65 tokens, 4096 x 256: fp32 274 us, bf16 at odd places 56; 64 tokens in few_any_kernel 69 and 29).
struct AnyPlan {
  int side;
  u32 splits;
};
AnyPlan any_plan(Product kind, const ProductLaunch& a, zero_dtype_t t) {
  AnyPlan best{128, 1};
  if (kind == kForward) return best;
  const int64_t halves = kind == kWeight ? 2 : 1, step = t == ZERO_F32 ? 32 : 64;
  const int64_t steps = (a.k + step - 1) / step * (kind == kInput ? 2 : 1), bytes = halves * a.rows * partial_cols(a.cols) * 4;
  double least = 1e300;
  for (int side : {128, 64}) {
    const int64_t tiles = (a.rows + side - 1) / side * ((a.cols + side - 1) / side) * halves, full = side == 128 ? 512 : 1024;
    const double alone = t == ZERO_F32 ? (side == 128 ? 2.2 : 0.8) : (side == 128 ? 1.0 : 0.7);
    const double shared = t == ZERO_F32 ? (side == 128 ? 4.2 : 2.4) : (side == 128 ? 1.45 : 1.0);
    for (u32 n = 1; n <= (t == ZERO_F32 ? kMaxSplits : kMaxSplits / 2); ++n) {
      if (n > 1 && (steps / n < 4 || bytes > kMaxPartialBytes / n)) break;
      const int64_t groups = tiles * n;
      double us = (groups <= 256 ? alone : shared * (double)((groups + full - 1) / full)) * (double)steps / n;
      if (n > 1) us += 3.0 + 2.0 * n * (double)bytes / 5e6;
      if (us < least) least = us, best = AnyPlan{side, n};
    }
  }
  return best;
}

template <class T, Product KIND, int SIDE>
int any_tiles(const ProductLaunch& a, u32 splits, hipStream_t s) {
  constexpr int cols = KIND == kForward ? SIDE / 2 : SIDE;
  const u32 down = (u32)((a.rows + SIDE - 1) / SIDE), across = (u32)((a.cols + cols - 1) / cols);
  hipLaunchKernelGGL((any_kernel<T, KIND, SIDE>), dim3(down * across * (KIND == kWeight ? 2 : 1) * splits), dim3(256), 0, s, a, down,
                     across, splits);
  return launched(KIND == kForward ? "gated projections" : KIND == kInput ? "gated input gradient" : "gated weight gradient");
}

template <class T, Product KIND>
int any_as(const ProductLaunch& a, zero_dtype_t t, hipStream_t s) {
  if constexpr (KIND == kForward) {
    if (a.rows <= 16) return few_any_as<T, 16>(a, s);
    if (a.rows <= 32) return few_any_as<T, 32>(a, s);
    if (a.rows <= 64) return few_any_as<T, 64>(a, s);
  }
  const AnyPlan plan = any_plan(KIND, a, t);
  if (int rc = KIND != kForward && plan.side == 64 ? any_tiles<T, KIND, KIND == kForward ? 128 : 64>(a, plan.splits, s)
                                                   : any_tiles<T, KIND, 128>(a, plan.splits, s))
    return rc;
  return plan.splits > 1 ? launch_join(KIND, a, t, plan.splits, s) : ZERO_OK;
}

template <Product KIND>
int any_of(const ProductLaunch& a, zero_dtype_t t, hipStream_t s) {
  switch (t) {
    case ZERO_F32: return any_as<F32, KIND>(a, t, s);
    case ZERO_BF16: return any_as<BF16, KIND>(a, t, s);
    default: return any_as<F16, KIND>(a, t, s);
  }
}

}  // namespace

int launch_product_any(Product kind, const ProductLaunch& a, zero_dtype_t t, void* stream) {
  const hipStream_t s = (hipStream_t)stream;
  return kind == kForward ? any_of<kForward>(a, t, s) : kind == kInput ? any_of<kInput>(a, t, s) : any_of<kWeight>(a, t, s);
}

int launch_join(Product kind, const ProductLaunch& a, zero_dtype_t t, u32 splits, void* stream) {
  const hipStream_t s = (hipStream_t)stream;
  if (kind == kWeight) return join_as<F32, kWeight>(a, splits, s);  // the results' type is a.out_type
  return t == ZERO_F32    ? join_as<F32, kInput>(a, splits, s)
         : t == ZERO_BF16 ? join_as<BF16, kInput>(a, splits, s)
                          : join_as<F16, kInput>(a, splits, s);
}

}  // namespace zk
