// HIP kernels for gfx950 (CDNA4): the model's input layer next to the sharded step --
// embedding lookup from the gather buffer, its gradient into a flat gradient
// buffer, and dropout from a counter-based generator.
//
// All three move far more bytes than they compute (a few flops per element), so
// none uses the matrix cores; what they need is wide accesses, enough of them in
// flight, and a generator cheap enough to hide behind them.  A lane's unit of work is
// one row's group of 8 columns: one 16-byte access of a 16-bit type, and one
// Philox4x32-10 call, whose 128 bits serve 8 elements with 16 bits each.
// Tensors sit anywhere in a flat buffer, so vectors are element aligned only;
// gfx950 takes 16-byte global accesses at any such address.
// Arithmetic is IEEE fp32, one rounding per operation (the build disables
// contraction); 16-bit results are rounded once, to nearest even.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdio>

#include "input.h"

namespace zk {
namespace {

using u32 = uint32_t;
using u64 = uint64_t;

struct F32 { static constexpr int bytes = 4; };
struct BF16 { static constexpr int bytes = 2; };
struct F16 { static constexpr int bytes = 2; };

typedef u32 vec4 __attribute__((ext_vector_type(4)));
typedef vec4 vec4_any __attribute__((aligned(2)));  // 16 bytes at an element-aligned address

// 8 elements, raw
template <class T>
struct Raw8 {
  vec4 q[T::bytes / 2];
};

template <class T>
__device__ __forceinline__ Raw8<T> load8(const char* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < T::bytes / 2; ++i) r.q[i] = *reinterpret_cast<const vec4_any*>(p + 16 * i);
  return r;
}

// the first n < 8 elements, zeros behind them
template <class T>
__device__ __forceinline__ Raw8<T> load_some(const char* p, u32 n) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < T::bytes / 2; ++i) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      u32 v = 0;
      if constexpr (T::bytes == 4) {
        const u32 e = 4 * i + w;
        if (e < n) v = reinterpret_cast<const u32*>(p)[e];
      } else {
        const u32 e = 2 * w;
        if (e < n) v = reinterpret_cast<const uint16_t*>(p)[e];
        if (e + 1 < n) v |= (u32) reinterpret_cast<const uint16_t*>(p)[e + 1] << 16;
      }
      r.q[i][w] = v;
    }
  }
  return r;
}

template <class T>
__device__ __forceinline__ void widen8(const Raw8<T>& r, float o[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (T::bytes == 4) {
      o[j] = __uint_as_float(r.q[j / 4][j % 4]);
    } else {
      const u32 w = r.q[0][j / 2];
      if constexpr (std::is_same<T, BF16>::value)
        o[j] = __uint_as_float(j % 2 ? (w & 0xffff0000u) : (w << 16));
      else
        o[j] = (float)__builtin_bit_cast(_Float16, (uint16_t)(j % 2 ? w >> 16 : w));
    }
  }
}

template <class T>
__device__ __forceinline__ u32 bits_of(float v) {
  if constexpr (T::bytes == 4) return __float_as_uint(v);
  else if constexpr (std::is_same<T, BF16>::value) return __builtin_bit_cast(uint16_t, (__bf16)v);
  else return __builtin_bit_cast(uint16_t, (_Float16)v);
}

template <class T>
__device__ __forceinline__ void store8(char* p, const float v[8]) {
#pragma unroll
  for (int i = 0; i < T::bytes / 2; ++i) {
    vec4 x;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if constexpr (T::bytes == 4) x[w] = bits_of<T>(v[4 * i + w]);
      else x[w] = bits_of<T>(v[2 * w]) | bits_of<T>(v[2 * w + 1]) << 16;
    }
    *reinterpret_cast<vec4_any*>(p + 16 * i) = x;
  }
}

template <class T>
__device__ __forceinline__ void store_some(char* p, const float v[8], u32 n) {
#pragma unroll
  for (u32 j = 0; j < 8; ++j) {
    if (j >= n) continue;
    if constexpr (T::bytes == 4) reinterpret_cast<float*>(p)[j] = v[j];
    else reinterpret_cast<uint16_t*>(p)[j] = (uint16_t)bits_of<T>(v[j]);
  }
}

template <class T>
__device__ __forceinline__ Raw8<T> load_n(const char* p, u32 n) {
  return n >= 8 ? load8<T>(p) : load_some<T>(p, n);
}
template <class T>
__device__ __forceinline__ void store_n(char* p, const float v[8], u32 n) {
  if (n >= 8) store8<T>(p, v);
  else store_some<T>(p, v, n);
}

__device__ __forceinline__ u32 quotient(u32 n, const FastDiv& f) { return (u32)(((u64)n * f.m) >> f.sh); }

// ---------------------------------------------------------------------------
// dropout's generator
// ---------------------------------------------------------------------------

// Philox4x32-10: ten rounds of two 32 x 32 -> 64 bit products (constants and
// round as published, Salmon et al., SC'11).  On CDNA a product with both halves is
// one quarter-rate instruction, so a call costs a wave about 10 * (2 * 16 + 4 * 4)
// cycles for 8 elements per lane.
__device__ __forceinline__ void philox(u32 c0, u32 c1, u32 c2, u32 c3, u32 k0, u32 k1, u32 w[4]) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const u64 a = (u64)c0 * 0xD2511F53u;
    const u64 b = (u64)c2 * 0xCD9E8D57u;
    c0 = (u32)(b >> 32) ^ c1 ^ k0;
    c2 = (u32)(a >> 32) ^ c3 ^ k1;
    c1 = (u32)b;
    c3 = (u32)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  w[0] = c0; w[1] = c1; w[2] = c2; w[3] = c3;
}

__device__ __forceinline__ u32 drop_step(const DropK& d) {
  return d.step_dev ? (u32)*d.step_dev : d.step;
}

// zeroes the dropped of the 8 values of (row, group); the kept are not scaled
__device__ __forceinline__ void drop8(const DropK& d, u32 step, u32 row, u32 group, float v[8]) {
  // The empty asm keeps the compiler from holding all twenty round keys in scalar
  // registers across calls (the gradient's unrolled loop ran out of them); two
  // scalar adds a round are free beside the vector multiplies.
  u32 k0 = d.key0, k1 = d.key1, w[4];
  asm volatile("" : "+s"(k0), "+s"(k1));
  philox(group, d.row0 + row, step, d.site, k0, k1, w);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = (w[j] & 0xffffu) >= d.thr ? v[2 * j] : 0.0f;
    v[2 * j + 1] = (w[j] >> 16) >= d.thr ? v[2 * j + 1] : 0.0f;
  }
}

// ---------------------------------------------------------------------------
// dropout
// ---------------------------------------------------------------------------

// Unit u = (row u / groups, group u % groups); a workgroup takes U * 256
// consecutive units, a lane U of them 256 apart, all loads before the arithmetic.
template <class XT, class OT, int U, bool DROP>
__global__ __launch_bounds__(kInThreads) void dropout_kernel(const DropoutLaunch a) {
  const u32 base = blockIdx.x * (u32)(kInThreads * U) + threadIdx.x;
  const u32 step = DROP ? drop_step(a.drop) : 0;
  u32 row[U], grp[U], n[U];
  Raw8<XT> x[U];
  Raw8<OT> r[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const u32 u = base + i * kInThreads;
    n[i] = 0;
    if (u >= a.units) continue;
    row[i] = quotient(u, a.groups);
    grp[i] = u - row[i] * a.groups.d;
    n[i] = a.cols - grp[i] * kGroup;
    x[i] = load_n<XT>(a.x + (int64_t)row[i] * a.ld_x + (int64_t)grp[i] * (kGroup * XT::bytes), n[i]);
    if (a.res) r[i] = load_n<OT>(a.res + (int64_t)row[i] * a.ld_res + (int64_t)grp[i] * (kGroup * OT::bytes), n[i]);
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    if (n[i] == 0) continue;
    float v[8];
    widen8<XT>(x[i], v);
    if constexpr (DROP) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= a.drop.ks;
      drop8(a.drop, step, row[i], grp[i], v);
    }
    if (a.res) {
      float o[8];
      widen8<OT>(r[i], o);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += o[j];
    }
    store_n<OT>(a.out + (int64_t)row[i] * a.ld_out + (int64_t)grp[i] * (kGroup * OT::bytes), v, n[i]);
  }
}

// ---------------------------------------------------------------------------
// embedding lookup
// ---------------------------------------------------------------------------

__device__ __forceinline__ int64_t id_at(const void* ids, int32_t id64, u32 t) {
  return id64 ? reinterpret_cast<const int64_t*>(ids)[t] : (int64_t) reinterpret_cast<const int32_t*>(ids)[t];
}

template <class TT, class OT, int U, bool DROP>
__global__ __launch_bounds__(kInThreads) void lookup_kernel(const LookupLaunch a) {
  const u32 base = blockIdx.x * (u32)(kInThreads * U) + threadIdx.x;
  const u32 step = DROP ? drop_step(a.drop) : 0;
  u32 row[U], grp[U], n[U];
  int64_t tab[U], pos[U];
  Raw8<TT> x[U], y[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const u32 u = base + i * kInThreads;
    n[i] = 0;
    tab[i] = pos[i] = -1;
    if (u >= a.units) continue;
    row[i] = quotient(u, a.groups);
    grp[i] = u - row[i] * a.groups.d;
    n[i] = a.dim - grp[i] * kGroup;
    tab[i] = id_at(a.ids, a.id64, row[i]);
    if (a.pos_table) {
      const u32 t = a.t0 + row[i];
      pos[i] = a.pos ? id_at(a.pos, a.id64, row[i]) : (int64_t)(t - quotient(t, a.period) * a.period.d);
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    if (n[i] == 0) continue;
    const int64_t col = (int64_t)grp[i] * (kGroup * TT::bytes);
    // unsigned: an id below id0, or so far from it that the difference wraps, is outside too
    const u64 v = (u64)tab[i] - (u64)a.id0;
    const bool in_tab = v < (u64)a.rows, in_pos = a.pos_table && (u64)pos[i] < (u64)a.pos_rows;
    x[i] = Raw8<TT>{};
    y[i] = Raw8<TT>{};
    if (in_tab) x[i] = load_n<TT>(a.table + (int64_t)v * a.ld_table + col, n[i]);
    if (in_pos) y[i] = load_n<TT>(a.pos_table + pos[i] * a.ld_pos + col, n[i]);
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    if (n[i] == 0) continue;
    float v[8];
    widen8<TT>(x[i], v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= a.scale;
    if (a.pos_table) {
      float o[8];
      widen8<TT>(y[i], o);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += o[j];
    }
    if constexpr (DROP) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= a.drop.ks;
      drop8(a.drop, step, a.t0 + row[i], grp[i], v);
    }
    store_n<OT>(a.out + (int64_t)row[i] * a.ld_out + (int64_t)grp[i] * (kGroup * OT::bytes), v, n[i]);
  }
}

// ---------------------------------------------------------------------------
// embedding gradient
// ---------------------------------------------------------------------------
//
// 1. sort_kernel orders the positions t by id (perm, and the row of each in
//    skey), equal ids by ascending t, and zeroes the rows without an id.
// 2. grad_sum_kernel cuts the order into tiles of equal length, so that a frequent
//    id is shared by many waves, and sums each run of equal ids inside a tile; a run that
//    crosses a tile border leaves an fp32 partial row instead of a result.
// 3. grad_join_kernel adds the partial rows of each such run, in order.
// No floating-point atomics: the same call gives the same bits.

// One workgroup per class c = row mod classes (frequent ids are neighbours in
// most vocabularies, so classes are interleaved).  Every workgroup reads all ids,
// counts those of lower classes -- which is where its own begin in the order --
// and places its own.  Nothing passes between workgroups.  Wave w owns a
// contiguous range of positions; cnt[w][k] first counts its ids of the class's
// row k, then holds the place of its next one.
__global__ __launch_bounds__(kSortThreads) void sort_kernel(const GradLaunch a, int fill_bytes) {
  extern __shared__ u32 cnt[];  // [kSortWaves][keys], then tot[keys]
  __shared__ u32 wave_sum[kSortWaves], lower_sum;
  const u32 cls = blockIdx.x, mask = (1u << a.lg_classes) - 1, keys = a.keys;
  const u32 lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  u32* const tot = cnt + kSortWaves * keys;
  for (u32 i = threadIdx.x; i < kSortWaves * keys; i += kSortThreads) cnt[i] = 0;
  if (threadIdx.x == 0) lower_sum = 0;
  __syncthreads();

  const u32 chunk = ((a.n + kSortThreads - 1) / kSortThreads) * 64;  // positions per wave, a multiple of 64
  const u32 t_lo = min(a.n, wave * chunk), t_hi = min(a.n, t_lo + chunk);
  u32* const mine = cnt + wave * keys;
  u32 lower = 0;
  for (u32 t0 = t_lo; t0 < t_hi; t0 += 64) {
    const u32 t = t0 + lane;
    u64 v = ~(u64)0;
    if (t < t_hi) v = (u64)id_at(a.ids, a.id64, t) - (u64)a.id0;
    const bool in = v < (u64)a.rows;
    const u32 c = (u32)v & mask;
    lower += (in && c < cls) ? 1 : 0;
    u64 own = __ballot(in && c == cls);
    const u32 k = (u32)v >> a.lg_classes;
    while (own) {  // one turn per distinct row
      const int l = __builtin_ctzll(own);
      const u32 kk = __builtin_amdgcn_readlane(k, l);
      const u64 same = __ballot(k == kk) & own;
      if ((int)lane == l) atomicAdd(&mine[kk], (u32)__popcll(same));
      own &= ~same;
    }
  }
  for (int o = 32; o; o >>= 1) lower += __shfl_xor(lower, o);
  if (lane == 0) atomicAdd(&lower_sum, lower);
  __syncthreads();

  // exclusive prefix over (row, wave); thread k owns row k
  u32 sum = 0;
  if (threadIdx.x < keys)
    for (int w = 0; w < kSortWaves; ++w) sum += cnt[w * keys + threadIdx.x];
  u32 incl = sum;
  for (int o = 1; o < 64; o <<= 1) {
    const u32 y = __shfl_up(incl, o);
    if ((int)lane >= o) incl += y;
  }
  if (lane == 63) wave_sum[wave] = incl;
  __syncthreads();
  u32 before = lower_sum, all = lower_sum;
  for (u32 w = 0; w < kSortWaves; ++w) {
    if (w < wave) before += wave_sum[w];
    all += wave_sum[w];
  }
  if (threadIdx.x < keys) {
    u32 at = before + incl - sum;
    for (int w = 0; w < kSortWaves; ++w) {
      const u32 x = cnt[w * keys + threadIdx.x];
      cnt[w * keys + threadIdx.x] = at;
      at += x;
    }
    tot[threadIdx.x] = sum;
  }
  if (cls == mask && threadIdx.x == 0) *a.n_valid = all;
  __syncthreads();

  for (u32 t0 = t_lo; t0 < t_hi; t0 += 64) {
    const u32 t = t0 + lane;
    u64 v = ~(u64)0;
    if (t < t_hi) v = (u64)id_at(a.ids, a.id64, t) - (u64)a.id0;
    u64 own = __ballot(v < (u64)a.rows && ((u32)v & mask) == cls);
    const u32 k = (u32)v >> a.lg_classes;
    while (own) {
      const int l = __builtin_ctzll(own);
      const u32 kk = __builtin_amdgcn_readlane(k, l);
      const u64 same = __ballot(k == kk) & own;
      u32 at = 0;
      if ((int)lane == l) at = atomicAdd(&mine[kk], (u32)__popcll(same));
      at = __builtin_amdgcn_readlane(at, l);
      if (same >> lane & 1) {
        at += (u32)__popcll(same & (((u64)1 << lane) - 1));
        a.perm[at] = t;
        a.skey[at] = (u32)v;
      }
      own &= ~same;
    }
  }

  if (a.accumulate) return;
  for (u32 k = wave; k < keys; k += kSortWaves) {
    const u64 row = ((u64)k << a.lg_classes) + cls;
    if (row >= (u64)a.rows || tot[k] != 0) continue;
    char* const p = a.grad + (int64_t)row * a.ld_grad;
    const float z[8] = {};
    for (u32 c = lane * 8; c < a.dim; c += 512) {
      if (fill_bytes == 4) store_n<F32>(p + (int64_t)c * 4, z, a.dim - c);
      else store_n<BF16>(p + (int64_t)c * 2, z, a.dim - c);
    }
  }
}

// zeroes the rows outside [row_lo, row_hi): one wave per row
__global__ __launch_bounds__(kInThreads) void fill_kernel(const GradLaunch a, int fill_bytes) {
  const u32 i = blockIdx.x * (kInThreads / 64) + (threadIdx.x >> 6);
  const u32 row = i < a.row_lo ? i : i - a.row_lo + a.row_hi;
  if ((int64_t)row >= a.rows) return;
  char* const p = a.grad + (int64_t)row * a.ld_grad;
  const float z[8] = {};
  for (u32 c = (threadIdx.x & 63) * 8; c < a.dim; c += 512) {
    if (fill_bytes == 4) store_n<F32>(p + (int64_t)c * 4, z, a.dim - c);
    else store_n<BF16>(p + (int64_t)c * 2, z, a.dim - c);
  }
}

// position p of the order: its t and its row
template <bool SORTED>
__device__ __forceinline__ void order_at(const GradLaunch& a, u32 p, u32& t, u32& row) {
  if constexpr (SORTED) {
    t = a.perm[p];
    row = a.skey[p];
  } else {
    p += a.start_lo;
    u32 id, i;
    if (p < a.split) {
      id = quotient(p, a.div_long);
      i = p - id * a.div_long.d;
    } else {
      p -= a.split;
      id = quotient(p, a.div_short);
      i = p - id * a.div_short.d;
      id += a.long_ids;
    }
    t = id + i * a.period;
    row = (u32)((int64_t)id - a.id0);
  }
}
template <bool SORTED>
__device__ __forceinline__ u32 row_at(const GradLaunch& a, u32 p) {
  u32 t, row;
  order_at<SORTED>(a, p, t, row);
  return row;
}

template <class GT>
__device__ __forceinline__ void write_row8(const GradLaunch& a, u32 row, u32 col, const float acc[8]) {
  char* const p = a.grad + (int64_t)row * a.ld_grad + (int64_t)col * GT::bytes;
  const u32 n = a.dim - col;
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = acc[j] * a.factor;
  if (a.accumulate) {
    float o[8];
    widen8<GT>(load_n<GT>(p, n), o);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += o[j];
  }
  store_n<GT>(p, v, n);
}

// rows of dy in flight per wave
template <bool DROP> constexpr int kSumBatch = DROP ? 4 : 8;

// One wave per (tile, 512 columns).
template <class DT, class GT, bool SORTED, bool DROP>
__global__ __launch_bounds__(kInThreads) void grad_sum_kernel(const GradLaunch a, u32 slabs) {
  const u32 lane = threadIdx.x & 63;
  const u32 w = __builtin_amdgcn_readfirstlane(blockIdx.x * (kInThreads / 64) + (threadIdx.x >> 6));
  const u32 tile = w / slabs, slab = w - tile * slabs;
  const u32 total = SORTED ? *a.n_valid : a.total;
  const u32 p0 = tile * a.tile;
  if (tile >= a.n_tiles || p0 >= total) return;
  const u32 n = min(a.tile, total - p0);
  const u32 group = slab * 64 + lane, col = group * kGroup;
  const u32 cols = col < a.dim ? a.dim - col : 0;
  const u32 step = DROP ? drop_step(a.drop) : 0;

  u32 t = 0, row = 0;
  if (lane < n) order_at<SORTED>(a, p0 + lane, t, row);
  const u32 next = __shfl_down(row, 1);
  const u64 ends = __ballot(lane + 1 == n || (lane + 1 < n && next != row));
  // does the first run continue from the tile before, the last one into the next?
  const u32 first_row = __builtin_amdgcn_readlane(row, 0), last_row = __builtin_amdgcn_readlane(row, n - 1);
  const bool from_left = p0 > 0 && row_at<SORTED>(a, p0 - 1) == first_row;
  const bool to_right = p0 + n < total && row_at<SORTED>(a, p0 + n) == last_row;

  float acc[8] = {};
  u32 run = 0;  // first position of the current run
  for (u32 i0 = 0; i0 < n; i0 += kSumBatch<DROP>) {
    Raw8<DT> x[kSumBatch<DROP>];
#pragma unroll
    for (int b = 0; b < kSumBatch<DROP>; ++b) {
      x[b] = Raw8<DT>{};
      if (i0 + b < n && cols) {
        const u32 tt = __builtin_amdgcn_readlane(t, i0 + b);
        x[b] = load_n<DT>(a.dy + (int64_t)tt * a.ld_dy + (int64_t)col * DT::bytes, cols);
      }
    }
#pragma unroll
    for (int b = 0; b < kSumBatch<DROP>; ++b) {
      const u32 i = i0 + b;
      if (i >= n) break;
      float v[8];
      widen8<DT>(x[b], v);
      if constexpr (DROP) drop8(a.drop, step, __builtin_amdgcn_readlane(t, i), group, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] += v[j];
      if (ends >> i & 1) {
        const bool left = run == 0 && from_left, right = i + 1 == n && to_right;
        if (cols) {
          if (left || right) {
            float* const q = a.partial + ((u64)tile * 2 + (left ? 0 : 1)) * a.ld_partial + col;
#pragma unroll
            for (int j = 0; j < 8; j += 4)
              *reinterpret_cast<float4*>(q + j) = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
          } else {
            write_row8<GT>(a, __builtin_amdgcn_readlane(row, i), col, acc);
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
        run = i + 1;
      }
    }
  }
}

// One workgroup per (tile in which a crossing run begins, 512 columns): the
// waves take consecutive parts of the run's tiles, wave 0 adds their sums.
template <class GT, bool SORTED>
__global__ __launch_bounds__(kJoinThreads) void grad_join_kernel(const GradLaunch a, u32 slabs) {
  constexpr u32 W = kJoinThreads / 64;
  __shared__ float part[W][64][8];
  const u32 tile = blockIdx.x / slabs, slab = blockIdx.x - tile * slabs;
  const u32 total = SORTED ? *a.n_valid : a.total;
  const u32 p1 = (tile + 1) * a.tile;
  if (p1 >= total) return;
  const u32 p0 = tile * a.tile;
  const u32 row = row_at<SORTED>(a, p1);
  if (row_at<SORTED>(a, p1 - 1) != row) return;
  if (p0 > 0 && row_at<SORTED>(a, p0) == row && row_at<SORTED>(a, p0 - 1) == row) return;  // began earlier
  // tiles (tile, last] begin with this row: a run is contiguous, so the first
  // tile that does not ends the search (64 tiles a turn)
  const u32 lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const u32 n_tiles = (total + a.tile - 1) / a.tile;
  u32 last = tile + 1;
  for (u32 c0 = tile + 2;; c0 += 64) {
    const u32 c = c0 + lane;
    const u64 other = __ballot(!(c < n_tiles && row_at<SORTED>(a, min(c, n_tiles - 1) * a.tile) == row));
    if (other) {
      last = c0 + (u32)__builtin_ctzll(other) - 1;
      break;
    }
  }
  const u32 m = last - tile, each = (m + W - 1) / W;
  const u32 lo = tile + 1 + min(m, wave * each), hi = min(last + 1, lo + each);
  const u32 col = (slab * 64 + lane) * kGroup;
  float acc[8] = {};
  if (col < a.dim)
#pragma unroll 4
    for (u32 c = lo; c < hi; ++c) {
      const float* const q = a.partial + (u64)c * 2 * a.ld_partial + col;
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] += q[j];
    }
#pragma unroll
  for (int j = 0; j < 8; ++j) part[wave][lane][j] = acc[j];
  __syncthreads();
  if (wave != 0 || col >= a.dim) return;
  const float* const q = a.partial + ((u64)tile * 2 + 1) * a.ld_partial + col;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    acc[j] = q[j];
    for (u32 w = 0; w < W; ++w) acc[j] += part[w][lane][j];
  }
  write_row8<GT>(a, row, col, acc);
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

int launched(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e == hipSuccess) return ZERO_OK;
  char buf[256];
  snprintf(buf, sizeof buf, "%s: HIP error %d (%s)", what, (int)e, hipGetErrorString(e));
  return fail(ZERO_EHIP, buf);
}

constexpr u32 kFewUnits = 256 * 256 * 4;  // below: one unit per lane, to spread the work over the CUs

template <class XT, class OT>
void dropout_as(const DropoutLaunch& a, hipStream_t st) {
  const dim3 b(kInThreads);
  const u32 per = a.units < kFewUnits ? kInThreads : 2 * kInThreads;
  const dim3 g((u32)(((u64)a.units + per - 1) / per));
  if (per == kInThreads) {
    if (a.drop.thr) hipLaunchKernelGGL((dropout_kernel<XT, OT, 1, true>), g, b, 0, st, a);
    else hipLaunchKernelGGL((dropout_kernel<XT, OT, 1, false>), g, b, 0, st, a);
  } else {
    if (a.drop.thr) hipLaunchKernelGGL((dropout_kernel<XT, OT, 2, true>), g, b, 0, st, a);
    else hipLaunchKernelGGL((dropout_kernel<XT, OT, 2, false>), g, b, 0, st, a);
  }
}

template <class TT, class OT>
void lookup_as(const LookupLaunch& a, hipStream_t st) {
  const dim3 b(kInThreads);
  const u32 per = a.units < kFewUnits ? kInThreads : 2 * kInThreads;
  const dim3 g((u32)(((u64)a.units + per - 1) / per));
  if (per == kInThreads) {
    if (a.drop.thr) hipLaunchKernelGGL((lookup_kernel<TT, OT, 1, true>), g, b, 0, st, a);
    else hipLaunchKernelGGL((lookup_kernel<TT, OT, 1, false>), g, b, 0, st, a);
  } else {
    if (a.drop.thr) hipLaunchKernelGGL((lookup_kernel<TT, OT, 2, true>), g, b, 0, st, a);
    else hipLaunchKernelGGL((lookup_kernel<TT, OT, 2, false>), g, b, 0, st, a);
  }
}

template <class DT, class GT, bool SORTED>
int grad_as(const GradLaunch& a, hipStream_t st) {
  const u32 slabs = (a.dim + 511) / 512;
  const int fill_bytes = GT::bytes;
  if constexpr (SORTED) {
    const size_t lds = (size_t)(kSortWaves + 1) * a.keys * sizeof(u32);
    hipLaunchKernelGGL(sort_kernel, dim3(1u << a.lg_classes), dim3(kSortThreads), lds, st, a, fill_bytes);
  } else if (!a.accumulate) {
    const int64_t rows = a.rows - (int64_t)(a.row_hi - a.row_lo);
    if (rows > 0)
      hipLaunchKernelGGL(fill_kernel, dim3((u32)((rows + 3) / 4)), dim3(kInThreads), 0, st, a, fill_bytes);
  }
  if (int rc = launched("embedding gradient")) return rc;
  if (a.n_tiles == 0) return ZERO_OK;
  const u64 waves = (u64)a.n_tiles * slabs;
  const dim3 g((u32)((waves + 3) / 4)), b(kInThreads);
  if (a.drop.thr) hipLaunchKernelGGL((grad_sum_kernel<DT, GT, SORTED, true>), g, b, 0, st, a, slabs);
  else hipLaunchKernelGGL((grad_sum_kernel<DT, GT, SORTED, false>), g, b, 0, st, a, slabs);
  if (int rc = launched("embedding gradient")) return rc;
  if (a.n_tiles > 1)
    hipLaunchKernelGGL((grad_join_kernel<GT, SORTED>), dim3((a.n_tiles - 1) * slabs), dim3(kJoinThreads), 0, st, a,
                       slabs);
  return launched("embedding gradient");
}

// calls f with the element types of the two codes
template <class F>
int with_types(zero_dtype_t x, zero_dtype_t y, F&& f) {
  auto second = [&](auto tx) {
    switch (y) {
      case ZERO_F32: return f(tx, F32{});
      case ZERO_BF16: return f(tx, BF16{});
      default: return f(tx, F16{});
    }
  };
  switch (x) {
    case ZERO_F32: return second(F32{});
    case ZERO_BF16: return second(BF16{});
    default: return second(F16{});
  }
}

}  // namespace

uint32_t grad_tile(int64_t n_ids, int64_t) {
  uint32_t r = 16;
  while (r < 64 && n_ids / r > 4096) r *= 2;
  return r;
}

int launch_dropout(const DropoutLaunch& a, zero_dtype_t xt, zero_dtype_t ot, void* stream) {
  return with_types(xt, ot, [&](auto x, auto o) {
    dropout_as<decltype(x), decltype(o)>(a, (hipStream_t)stream);
    return launched("dropout");
  });
}

int launch_lookup(const LookupLaunch& a, zero_dtype_t tt, zero_dtype_t ot, void* stream) {
  return with_types(tt, ot, [&](auto t, auto o) {
    lookup_as<decltype(t), decltype(o)>(a, (hipStream_t)stream);
    return launched("embedding lookup");
  });
}

int launch_embed_grad(const GradLaunch& a, zero_dtype_t dt, zero_dtype_t gt, void* stream) {
  return with_types(dt, gt, [&](auto d, auto g) {
    if (a.ids) return grad_as<decltype(d), decltype(g), true>(a, (hipStream_t)stream);
    return grad_as<decltype(d), decltype(g), false>(a, (hipStream_t)stream);
  });
}

}  // namespace zk
