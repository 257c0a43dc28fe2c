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
// Results are stored non-temporally: they are read by another kernel, if at all,
// and leave the L2 to what is read again (8192 x 1600 bf16, dropout with residual,
// 13.6 us against 15.5; lookup of 32768 rows of 4096, 79 against 85).
// Figures here are of one MI355X, calls back to back from a graph on four sets of inputs,
// where not said otherwise; a plain streaming copy of 2 GiB moves 6.6 TB/s there.
// "Vector units" is the share of the cycles in which a kernel runs that its vector
// instructions take at four cycles each.
// Arithmetic is IEEE fp32, one rounding per operation (the build disables
// contraction); 16-bit results are rounded once, to nearest even.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "elements.h"
#include "input.h"

namespace zk {
namespace {

// How the 64 lanes of a wave share 64 consecutive 8-column groups.  Two 16-bit
// tensors: lane l takes group l, 16 bytes.  With an fp32 tensor that would be 32
// bytes a lane, of which each 16-byte access of the wave touches every second half of a cache
// line; there lane l takes 4 columns, half l % 2 of group l / 2, and the same of
// group 32 + l / 2: every access of the wave is contiguous again.
template <class A, class B>
constexpr int kWidth = (A::bytes == 4 || B::bytes == 4) ? 4 : 8;  // columns of one piece; 8 / kWidth pieces
template <int W>
__device__ __forceinline__ u32 piece_group(u32 lane, int piece) {
  return W == 8 ? lane : (lane >> 1) + 32 * piece;
}
// of a value per piece, the one of the piece whose group the lane draws numbers for
template <int P>
__device__ __forceinline__ u32 own_piece(u32 lane, const u32 (&v)[P]) {
  const u32 first = v[0], last = v[P - 1];
  return P == 2 && (lane & 1) ? last : first;
}
template <int W>
__device__ __forceinline__ u32 piece_col(u32 lane) {  // first column within the group
  return W == 8 ? 0 : (lane & 1) * 4;
}

// (row, group) of unit u0 + i, for i < 64 and the wave's first unit u0 in row `first`.
// ONE: a row's groups are a multiple of 64, so the wave has one row, and what belongs
// to it is found once by scalar instructions rather than by every lane.
struct Unit {
  u32 row, grp;
};
template <bool ONE>
__device__ __forceinline__ Unit unit_at(u32 u0, u32 i, u32 first, const FastDiv& groups) {
  const u32 row = ONE ? first : quotient(u0 + i, groups);
  return Unit{row, u0 + i - row * groups.d};
}

// ---------------------------------------------------------------------------
// dropout's generator
// ---------------------------------------------------------------------------

// one instruction on gfx950 (truth table 0x96)
__device__ __forceinline__ u32 xor3(u32 a, u32 b, u32 c) { return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96); }

// Philox4x32-10: ten rounds of two 32 x 32 -> 64 bit products (constants and
// round as published, Salmon et al., SC'11).  A product with both halves is one
// instruction.  A call costs a wave 205 cycles of its SIMD for 8 elements per lane
// (measured with nothing else running; 124 with additions in the products' place).
__device__ __forceinline__ void philox(u32 c0, u32 c1, u32 c2, u32 c3, u32 k0, u32 k1, u32 w[4]) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const u64 a = (u64)c0 * 0xD2511F53u;
    const u64 b = (u64)c2 * 0xCD9E8D57u;
    c0 = xor3((u32)(b >> 32), c1, k0);
    c2 = xor3((u32)(a >> 32), c3, k1);
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

// The random words of a lane's 8 values.  (row, group) is the group whose numbers this
// lane computes: its own (W = 8), or that of piece lane % 2 (W = 4), where the two
// lanes of a pair hold half of each group and exchange two words.  Every lane of the
// wave has to take part.  Drawn after the loads of the values are issued and before they are used,
// the words cost little time of their own.
struct Words {
  u32 w[4];
};
template <int W>
__device__ __forceinline__ Words draw(const DropK& d, u32 step, u32 row, u32 group) {
  // The empty asm keeps the compiler from holding all twenty round keys in scalar
  // registers across calls (the gradient's unrolled loop ran out of them); two
  // scalar adds a round are free beside the vector multiplies.
  u32 k0 = d.key0, k1 = d.key1;
  asm volatile("" : "+s"(k0), "+s"(k1));
  Words r;
  philox(group, d.row0 + row, step, d.site, k0, k1, r.w);
  if constexpr (W == 4) {
    const bool odd = threadIdx.x & 1;
    // to the other lane of the pair: quad_perm [1, 0, 3, 2]
    const u32 a = __builtin_amdgcn_mov_dpp((int)(odd ? r.w[0] : r.w[2]), 0xB1, 0xF, 0xF, true);
    const u32 b = __builtin_amdgcn_mov_dpp((int)(odd ? r.w[1] : r.w[3]), 0xB1, 0xF, 0xF, true);
    if (odd) {
      r.w[0] = a;
      r.w[1] = b;
    } else {
      r.w[2] = a;
      r.w[3] = b;
    }
  }
  return r;
}
// zeroes the dropped among the values; the kept are not scaled
__device__ __forceinline__ void drop8(const DropK& d, const Words& r, float v[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = (r.w[j] & 0xffffu) >= d.thr ? v[2 * j] : 0.0f;
    v[2 * j + 1] = (r.w[j] >> 16) >= d.thr ? v[2 * j + 1] : 0.0f;
  }
}

// whether the one element (row, col) is kept
__device__ __forceinline__ bool kept(const DropK& d, u32 row, u32 col) {
  if (d.thr == 0) return true;
  u32 w[4];
  philox(col / kGroup, d.row0 + row, drop_step(d), d.site, d.key0, d.key1, w);
  const u32 j = col % kGroup / 2, u = j == 0 ? w[0] : j == 1 ? w[1] : j == 2 ? w[2] : w[3];
  return (col % 2 ? u >> 16 : u & 0xffffu) >= d.thr;
}

// Tensors of fewer than 8 elements are too short for the vector accesses of the
// kernels below; the *_short_kernels serve them element by element.

// ---------------------------------------------------------------------------
// dropout
// ---------------------------------------------------------------------------

__global__ void dropout_short_kernel(const DropoutLaunch a, int xt, int ot) {
  for (u64 i = threadIdx.x; i < (u64)a.rows * a.cols; i += blockDim.x) {
    const u32 r = (u32)(i / a.cols), c = (u32)(i % a.cols);
    float v = load_one(a.x + r * a.ld_x + (int64_t)c * one_bytes(xt), xt) * a.drop.ks;
    if (!kept(a.drop, r, c)) v = 0.0f;
    if (a.res) v += load_one(a.res + r * a.ld_res + (int64_t)c * one_bytes(ot), ot);
    store_one(a.out + r * a.ld_out + (int64_t)c * one_bytes(ot), ot, v);
  }
}

// A unit is (row, 8-column group), numbered row by row; a wave takes 64 consecutive ones.
// Bound by HBM: 8192 x 1600 bf16 with residual 12.4 us (6.4 TB/s, vector units 69%),
// 16384 x 4097 fp32 91 us (5.9 TB/s, 41%).
template <class XT, class OT, bool DROP, bool ONE>
__global__ __launch_bounds__(kInThreads) void dropout_kernel(const DropoutLaunch a) {
  constexpr int W = kWidth<XT, OT>, P = 8 / W;
  const u32 lane = threadIdx.x & 63;
  const u32 u0 = __builtin_amdgcn_readfirstlane(blockIdx.x * (u32)kInThreads + (threadIdx.x & ~63u));
  const u32 first = quotient(u0, a.groups);
  const u32 step = DROP ? drop_step(a.drop) : 0;
  u32 row[P], grp[P], n[P], dx[P], dr[P];
  Raw<XT, W> x[P];
  Raw<OT, W> r[P];
#pragma unroll
  for (int q = 0; q < P; ++q) {
    const Unit w = unit_at<ONE>(u0, piece_group<W>(lane, q), first, a.groups);
    row[q] = w.row;
    grp[q] = w.grp;
    const u32 col = w.grp * kGroup + piece_col<W>(lane);
    n[q] = u0 + piece_group<W>(lane, q) < a.units && col < a.cols ? a.cols - col : 0;
    dx[q] = dr[q] = 0;
    if (n[q] == 0) continue;
    dx[q] = load_w<XT, W>(a.x + (int64_t)w.row * a.ld_x + (int64_t)col * XT::bytes, a.x_end, x[q]);
    if (a.res) dr[q] = load_w<OT, W>(a.res + (int64_t)w.row * a.ld_res + (int64_t)col * OT::bytes, a.res_end, r[q]);
  }
  Words random{};
  if constexpr (DROP) random = draw<W>(a.drop, step, own_piece<P>(lane, row), own_piece<P>(lane, grp));
  float v[8];
#pragma unroll
  for (int q = 0; q < P; ++q) {
    move_down<XT, W>(x[q], dx[q]);
    widen<XT, W>(x[q], v + q * W);
  }
  if constexpr (DROP) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= a.drop.ks;
    drop8(a.drop, random, v);
  }
#pragma unroll
  for (int q = 0; q < P; ++q) {
    if (n[q] == 0) continue;
    if (a.res) {
      float o[W];
      move_down<OT, W>(r[q], dr[q]);
      widen<OT, W>(r[q], o);
#pragma unroll
      for (int j = 0; j < W; ++j) v[q * W + j] += o[j];
    }
    const u32 col = grp[q] * kGroup + piece_col<W>(lane);
    store_n<OT, W>(a.out + (int64_t)row[q] * a.ld_out + (int64_t)col * OT::bytes, v + q * W, n[q]);
  }
}

// ---------------------------------------------------------------------------
// embedding lookup
// ---------------------------------------------------------------------------

// Without a branch on the id's width: its low word, and its high word or the low
// one again, of which the sign is then the high word.
__device__ __forceinline__ int64_t id_at(const void* ids, int32_t id64, u32 t) {
  const u32* const p = reinterpret_cast<const u32*>(ids) + ((u64)t << id64);
  const u32 lo = p[0], hi = p[id64];
  return (int64_t)((u64)(id64 ? hi : (u32)((int32_t)hi >> 31)) << 32 | lo);
}

__device__ __forceinline__ int64_t pos_at(const LookupLaunch& a, u32 i) {
  const u32 t = a.t0 + i;
  return a.pos ? id_at(a.pos, a.id64, i) : (int64_t)(t - quotient(t, a.period) * a.period.d);
}

__global__ void lookup_short_kernel(const LookupLaunch a, int tt, int ot) {
  for (u64 i = (u64)blockIdx.x * blockDim.x + threadIdx.x; i < (u64)a.n * a.dim; i += (u64)gridDim.x * blockDim.x) {
    const u32 t = (u32)(i / a.dim), c = (u32)(i % a.dim);
    const u64 row = (u64)id_at(a.ids, a.id64, t) - (u64)a.id0;
    const int64_t col = (int64_t)c * one_bytes(tt);
    float v = (row < (u64)a.rows ? load_one(a.table + (int64_t)row * a.ld_table + col, tt) : 0.0f) * a.scale;
    if (a.pos_table) {
      const int64_t pos = pos_at(a, t);
      v += (u64)pos < (u64)a.pos_rows ? load_one(a.pos_table + pos * a.ld_pos + col, tt) : 0.0f;
    }
    v *= a.drop.ks;
    if (!kept(a.drop, a.t0 + t, c)) v = 0.0f;
    store_one(a.out + t * a.ld_out + (int64_t)c * one_bytes(ot), ot, v);
  }
}

// As above, with U times 64 units a wave, 256 apart, all loads before the arithmetic.
// 32768 of 128256 rows of 4096 bf16: 66 us.  Its 371 MB would take 56 us at the copy's
// rate; the eight L2 caches between them fetch the frequent rows again, 450 MB in all,
// which it moves at 6.8 TB/s.  8192 x 1600 bf16 with positions and dropout: 10.7
// us for 41 MB, bound by the vector units (95%): 212 instructions a wave, of which
// the generator has about a quarter; the rest finds rows, columns and tails,
// widens, scales and rounds.
template <class TT, class OT, int U, bool DROP, bool ONE>
__global__ __launch_bounds__(kInThreads) void lookup_kernel(const LookupLaunch a) {
  constexpr int W = kWidth<TT, OT>, P = 8 / W;
  const u32 lane = threadIdx.x & 63;
  const u32 base = __builtin_amdgcn_readfirstlane(blockIdx.x * (u32)(kInThreads * U) + (threadIdx.x & ~63u));
  const u32 step = DROP ? drop_step(a.drop) : 0;
  u32 row[U][P], grp[U][P], n[U][P], dx[U][P], dy[U][P];
  const char* tab[U][P];  // the table's row, or null
  const char* pos[U][P];
  Raw<TT, W> x[U][P], y[U][P];
  // unsigned: an id below id0, or so far from it that the difference wraps, is outside too
  auto table_row = [&](u32 t) -> const char* {
    const u64 v = (u64)id_at(a.ids, a.id64, min(t, a.n - 1)) - (u64)a.id0;
    return v < (u64)a.rows ? a.table + (int64_t)v * a.ld_table : nullptr;
  };
  auto pos_row = [&](u32 t) -> const char* {
    const u64 v = (u64)pos_at(a, min(t, a.n - 1));
    return v < (u64)a.pos_rows ? a.pos_table + (int64_t)v * a.ld_pos : nullptr;
  };
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const u32 u0 = base + i * kInThreads, first = quotient(u0, a.groups);
    const char *t0 = nullptr, *p0 = nullptr;
    if constexpr (ONE) {
      t0 = table_row(first);
      if (a.pos_table) p0 = pos_row(first);
    }
#pragma unroll
    for (int q = 0; q < P; ++q) {
      const Unit w = unit_at<ONE>(u0, piece_group<W>(lane, q), first, a.groups);
      row[i][q] = w.row;
      grp[i][q] = w.grp;
      const u32 col = w.grp * kGroup + piece_col<W>(lane);
      n[i][q] = u0 + piece_group<W>(lane, q) < a.units && col < a.dim ? a.dim - col : 0;
      pos[i][q] = nullptr;
      if constexpr (ONE) {
        tab[i][q] = t0;
        pos[i][q] = p0;
      } else {
        tab[i][q] = table_row(w.row);
        if (a.pos_table) pos[i][q] = pos_row(w.row);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i)
#pragma unroll
    for (int q = 0; q < P; ++q) {
      x[i][q] = Raw<TT, W>{};
      y[i][q] = Raw<TT, W>{};
      dx[i][q] = dy[i][q] = 0;
      const int64_t col = (int64_t)(grp[i][q] * kGroup + piece_col<W>(lane)) * TT::bytes;
      if (n[i][q] != 0 && tab[i][q]) dx[i][q] = load_w<TT, W>(tab[i][q] + col, a.table_end, x[i][q]);
      if (n[i][q] != 0 && pos[i][q]) dy[i][q] = load_w<TT, W>(pos[i][q] + col, a.pos_end, y[i][q]);
    }
  Words random[U];
  if constexpr (DROP) {
#pragma unroll
    for (int i = 0; i < U; ++i)
      random[i] = draw<W>(a.drop, step, a.t0 + own_piece<P>(lane, row[i]), own_piece<P>(lane, grp[i]));
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    float v[8];
#pragma unroll
    for (int q = 0; q < P; ++q) {
      move_down<TT, W>(x[i][q], dx[i][q]);
      widen<TT, W>(x[i][q], v + q * W);
#pragma unroll
      for (int j = 0; j < W; ++j) v[q * W + j] *= a.scale;
      if (a.pos_table) {
        float o[W];
        move_down<TT, W>(y[i][q], dy[i][q]);
        widen<TT, W>(y[i][q], o);
#pragma unroll
        for (int j = 0; j < W; ++j) v[q * W + j] += o[j];
      }
    }
    if constexpr (DROP) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= a.drop.ks;
      drop8(a.drop, random[i], v);
    }
#pragma unroll
    for (int q = 0; q < P; ++q) {
      if (n[i][q] == 0) continue;
      const u32 col = grp[i][q] * kGroup + piece_col<W>(lane);
      store_n<OT, W>(a.out + (int64_t)row[i][q] * a.ld_out + (int64_t)col * OT::bytes, v + q * W, n[i][q]);
    }
  }
}

// ---------------------------------------------------------------------------
// embedding gradient
// ---------------------------------------------------------------------------
//
// 1. sort_kernel orders the positions t by row, equal rows by ascending t.  Each
//    place of the order gets (t, row, its index within the row's run, the run's
//    length); each row a flag that says whether it has any.
// 2. grad_sum_kernel sums the runs in chunks of 1 << a.lg_chunk places, so that a frequent id
//    is shared by many waves.  A run of one chunk gives its row of the gradient,
//    the chunks of longer ones give fp32 partial rows.  Further workgroups of the
//    same launch zero the rows without an id.
// 3. grad_join_kernel adds the partial rows of each longer run, in order.
// No floating-point atomics: the same call gives the same bits.
// The smallest calls take one launch instead (grad_once_kernel).
//
// The gradient is mostly a write: 8192 ids into 50257 x 1600 bf16 move 187 MB, of
// which 161 MB are the result, and take 36.4 us, 28.4 at the copy's rate: 9 us order (37.7 MB
// of zero rows beside it), 24 us sums, 4 us joins.  65536 ids into 128256 x 4096 bf16
// (1.59 GB): 316 us, 241 at the copy's rate: 41 us order (125.8 MB of zero rows), 265 us
// sums at 5.6 TB/s, 9 us joins.  Added to what the gradient holds, where only the rows
// with an id move, they take 29.8 us for 50 MB (8, 18.5 and 4) and 228 us for 883 MB
// (25, 194 and 9.5).

// The row of position t's id, or kNoRow.
constexpr u32 kNoRow = ~0u;
__device__ __forceinline__ u32 row_of_id(const GradLaunch& a, u64 id) {
  const u64 v = id - (u64)a.id0;
  return v < (u64)a.rows ? (u32)v : kNoRow;
}

// Zeroes unit u, 0 <= u < a.fill_units.d, of the row at p: 16 bytes, counted from the
// multiple of a.fill_align at or before p.  For long rows that is a cache line, so that
// the lanes that share one write it whole (31216 rows of 8109 fp32: 206 us, 242
// counted from the rows' odd beginnings); short ones are counted from p itself.  At
// the row's ends, what is the row's.
template <class GT>
__device__ __forceinline__ void zero_unit(const GradLaunch& a, char* p, u32 u) {
  char* const end = p + (int64_t)a.dim * GT::bytes;
  char* const q = p - ((uintptr_t)p & (a.fill_align - 1)) + (int64_t)u * 16;
  if (q >= p && q + 16 <= end) {
    const vec4 z = {0, 0, 0, 0};
    __builtin_nontemporal_store(z, reinterpret_cast<vec4_any*>(q));
  } else {
#pragma unroll
    for (int j = 0; j < 16; j += GT::bytes) {
      char* const e = q + j;
      if (e < p || e >= end) continue;
      if constexpr (GT::bytes == 4) *reinterpret_cast<u32*>(e) = 0;
      else *reinterpret_cast<uint16_t*>(e) = 0;
    }
  }
}

// The places of class c = row mod classes in the order, found by one workgroup
// (frequent ids are neighbours in most vocabularies, so classes are interleaved).
// Every workgroup reads all ids, counts those of lower classes -- which is where its
// own begin in the order -- and lists its own.  Nothing passes between workgroups.
// Wave w owns a contiguous range of positions; cnt[w][k] first counts its ids of
// the class's row k, then holds the place of its next one.  The scan is a compare
// and a ballot per 64 ids; the few own ones go to a list, and counting and placing
// run over that.  By itself 8 us for 8192 ids and 25 us for 65536 (vector units 33
// and 55%).
//   lds: cnt[kSortWaves][keys], start[keys] (the first place of row k), tot[keys] (its
//        ids), lists [kSortWaves][a.list]
// Calls counted(first place of the class, first place behind it) between the two
// parts, with start and tot written but not yet seen by all waves, and then
// emit(place, position, row of the class) for each id of the class.
template <class Counted, class Emit>
__device__ __forceinline__ void order_class(const GradLaunch& a, u32 cls, u32* cnt, Counted&& counted, Emit&& emit) {
  __shared__ u32 wave_sum[kSortWaves], lower_sum;
  const u32 mask = (1u << a.lg_classes) - 1, keys = a.keys;
  const u32 lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  u32* const start = cnt + kSortWaves * keys;
  u32* const tot = start + keys;
  u32* const list = tot + keys + wave * a.list;  // (position - t_lo) << 10 | row of the class
  for (u32 i = threadIdx.x; i < kSortWaves * keys; i += kSortThreads) cnt[i] = 0;
  if (threadIdx.x == 0) lower_sum = 0;
  __syncthreads();

  const u32 chunk = ((a.n + kSortThreads - 1) / kSortThreads) * 64;  // positions per wave, a multiple of 64
  const u32 t_lo = min(a.n, wave * chunk), t_hi = min(a.n, t_lo + chunk);
  u32* const mine = cnt + wave * keys;

  // calls f(first position, row) for 64 positions at a time, in batches of
  // kSortAhead whose loads are issued a batch ahead
  auto scan_as = [&](auto zero, auto&& f) {
    using Id = decltype(zero);
    const Id* const ids = reinterpret_cast<const Id*>(a.ids);
    constexpr u32 B = 64 * kSortAhead;
    Id next[kSortAhead];
    auto fetch = [&](u32 t0) {
#pragma unroll
      for (u32 j = 0; j < kSortAhead; ++j) next[j] = ids[min(t0 + 64 * j + lane, a.n - 1)];
    };
    if (t_lo < t_hi) fetch(t_lo);
    for (u32 t0 = t_lo; t0 < t_hi; t0 += B) {
      Id id[kSortAhead];
#pragma unroll
      for (u32 j = 0; j < kSortAhead; ++j) id[j] = next[j];
      if (t0 + B < t_hi) fetch(t0 + B);
#pragma unroll
      for (u32 j = 0; j < kSortAhead; ++j) {
        const u32 t = t0 + 64 * j;
        if (t >= t_hi) break;
        const u32 row = row_of_id(a, (u64)(int64_t)id[j]);
        f(t, t + lane < t_hi ? row : kNoRow);
      }
    }
  };
  auto scan = [&](auto&& f) {
    if (a.id64) scan_as(int64_t{}, f);
    else scan_as(int32_t{}, f);
  };
  // calls f(leader lane, row k, its lanes) for each distinct k of the lanes in `own`
  auto each_row = [&](u64 own, u32 k, auto&& f) {
    while (own) {
      const int l = __builtin_ctzll(own);
      const u32 kk = __builtin_amdgcn_readlane(k, l);
      const u64 same = __ballot(k == kk) & own;
      f(l, kk, same);
      own &= ~same;
    }
  };
  auto below = [&](u64 m) { return (u32)__popcll(m & (((u64)1 << lane) - 1)); };

  u32 lower = 0, listed = 0;  // wave-uniform
  scan([&](u32 t, u32 row) {
    const u32 c = row & mask;
    const u64 in = __ballot(row != kNoRow);
    lower += (u32)__popcll(__ballot(c < cls) & in);
    const u64 own = __ballot(c == cls) & in;
    if (own == 0) return;
    const u32 at = listed + below(own);
    listed += (u32)__popcll(own);
    if ((own >> lane & 1) && at < a.list) list[at] = (t + lane - t_lo) << 10 | row >> a.lg_classes;
  });
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the list is read by other lanes of the wave
  // calls f(own lanes, position, row of the class) for the wave's own positions in
  // order, from its list or, where that is too short, from the ids again
  auto own_positions = [&](auto&& f) {
    if (listed <= a.list) {
      for (u32 i = 0; i < listed; i += 64) {
        const bool in = i + lane < listed;
        const u32 e = in ? list[i + lane] : 0;
        f(__ballot(in), t_lo + (e >> 10), e & 1023);
      }
    } else {
      scan([&](u32 t, u32 row) {
        const u64 own = __ballot(row != kNoRow && (row & mask) == cls);
        if (own) f(own, t + lane, row >> a.lg_classes);
      });
    }
  };
  own_positions([&](u64 own, u32, u32 k) {
    each_row(own, k, [&](int l, u32 kk, u64 same) {
      if ((int)lane == l) atomicAdd(&mine[kk], (u32)__popcll(same));
    });
  });
  if (lane == 0) atomicAdd(&lower_sum, lower);
  __syncthreads();

  // exclusive prefix over (row, wave); thread k owns row k
  u32 sum = 0, of_wave[kSortWaves];
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) {
    of_wave[w] = threadIdx.x < keys ? cnt[w * keys + threadIdx.x] : 0;
    sum += of_wave[w];
  }
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
    start[threadIdx.x] = at;
    tot[threadIdx.x] = sum;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      cnt[w * keys + threadIdx.x] = at;
      at += of_wave[w];
    }
  }
  counted(lower_sum, all);
  __syncthreads();

  own_positions([&](u64 own, u32 t, u32 k) {
    each_row(own, k, [&](int l, u32 kk, u64 same) {
      u32 at = 0;
      if ((int)lane == l) at = atomicAdd(&mine[kk], (u32)__popcll(same));
      at = __builtin_amdgcn_readlane(at, l) + below(same);
      if (same >> lane & 1) emit(at, t, kk);
    });
  });
}

// One workgroup per class.  That reads little and takes 8 to 25 us (8192 to 65536
// ids), so further workgroups of the launch zero the rows from a.early_row on
// meanwhile, whether they have ids or not: those that do are written again by the launches
// that follow.  With them the launch takes 9 to 41 us.
template <class GT>
__global__ __launch_bounds__(kSortThreads) void sort_kernel(const GradLaunch a) {
  if (blockIdx.x >> a.lg_classes) {
    const u32 r0 = a.early_row + (blockIdx.x - (1u << a.lg_classes)) * a.early_rows;
    const u32 per_row = a.fill_units.d, units = min(a.early_rows, (u32)a.rows - r0) * per_row;
    for (u32 u = threadIdx.x; u < units; u += kSortThreads) {
      const u32 i = quotient(u, a.fill_units);
      zero_unit<GT>(a, a.grad + (int64_t)(r0 + i) * a.ld_grad, u - i * per_row);
    }
    return;
  }
  extern __shared__ u32 lds[];
  const u32 cls = blockIdx.x, *const start = lds + kSortWaves * a.keys, *const tot = start + a.keys;
  order_class(
      a, cls, lds,
      [&](u32, u32 behind) {
        const u64 row = ((u64)threadIdx.x << a.lg_classes) + cls;
        if (threadIdx.x < a.keys && row < (u64)a.rows) a.has[row] = tot[threadIdx.x] != 0;
        if (cls + 1 == 1u << a.lg_classes && threadIdx.x == 0) *a.n_valid = behind;
      },
      [&](u32 at, u32 t, u32 k) {
        a.order[at] = make_uint4(t, (k << a.lg_classes) + cls, at - start[k], tot[k]);
      });
}

// dy of fewer than 8 elements, and so fewer than 8 ids: element by element
__global__ void grad_short_kernel(const GradLaunch a, int dt, int gt) {
  for (u64 i = (u64)blockIdx.x * blockDim.x + threadIdx.x; i < (u64)a.rows * a.dim; i += (u64)gridDim.x * blockDim.x) {
    const u32 row = (u32)(i / a.dim), c = (u32)(i % a.dim);
    float sum = 0.0f;
    bool any = false;
    for (u32 t = 0; t < a.n; ++t) {
      const u64 id = a.ids ? (u64)id_at(a.ids, a.id64, t) : t % a.period;
      if (row_of_id(a, id) != row) continue;
      any = true;
      if (kept(a.drop, t, c)) sum += load_one(a.dy + t * a.ld_dy + (int64_t)c * one_bytes(dt), dt);
    }
    char* const p = a.grad + (int64_t)row * a.ld_grad + (int64_t)c * one_bytes(gt);
    if (any) sum *= a.factor;  // else +0, whatever the factor's sign
    if (a.accumulate) {
      if (!any) continue;
      sum += load_one(p, gt);
    }
    store_one(p, gt, sum);
  }
}

// place p of the order: (t, row, index within the run, length of the run)
template <bool SORTED>
__device__ __forceinline__ uint4 order_at(const GradLaunch& a, u32 p) {
  if constexpr (SORTED) {
    return a.order[p];
  } else {
    p += a.start_lo;
    u32 id, i, len = a.div_short.d;
    if (p < a.split) {
      id = quotient(p, a.div_long);
      i = p - id * a.div_long.d;
      len = a.div_long.d;
    } else {
      p -= a.split;
      id = quotient(p, a.div_short);
      i = p - id * a.div_short.d;
      id += a.long_ids;
    }
    return make_uint4(id + i * a.period, (u32)((int64_t)id - a.id0), i, len);
  }
}

// Where the partial row of the chunk that begins at place p lies: at most one
// full chunk and the shorter tail of one other run begin in 1 << a.lg_chunk aligned places.
__device__ __forceinline__ u32 partial_slot(const GradLaunch& a, u32 p, bool tail) {
  return 2 * (p >> a.lg_chunk) + (tail ? 1 : 0);
}

// Writes a lane's sums, times the factor, to its columns of a row.
template <class GT, int W>
__device__ __forceinline__ void write_row8(const GradLaunch& a, u32 row, u32 slab, u32 lane, const float acc[8],
                                           float factor) {
#pragma unroll
  for (int q = 0; q < 8 / W; ++q) {
    const u32 col = (slab * 64 + piece_group<W>(lane, q)) * kGroup + piece_col<W>(lane);
    if (col >= a.dim) continue;
    char* const p = a.grad + (int64_t)row * a.ld_grad + (int64_t)col * GT::bytes;
    const u32 n = a.dim - col;
    float v[W];
#pragma unroll
    for (int j = 0; j < W; ++j) v[j] = acc[q * W + j] * factor;
    if (a.accumulate) {
      constexpr int type = std::is_same<GT, F32>::value ? ZERO_F32 : std::is_same<GT, BF16>::value ? ZERO_BF16 : ZERO_F16;
      if (n >= W) {
        Raw<GT, W> old;
        float o[W];
        load_w<GT, W>(p, p + W * GT::bytes, old);
        widen<GT, W>(old, o);
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] += o[j];
      } else {
#pragma unroll
        for (u32 j = 0; j < W; ++j)
          if (j < n) v[j] += load_one(p + j * GT::bytes, type);
      }
    }
    store_n<GT, W>(p, v, n);
  }
}

// Zeroes those of a.fill_rows rows from row r0 on that have no id.
template <class GT, bool SORTED>
__device__ __forceinline__ void fill_rows(const GradLaunch& a, u32 r0) {
  __shared__ uint8_t rows[64];
  const u32 lane = threadIdx.x & 63, row = r0 + lane;
  bool empty = lane < a.fill_rows && row < (SORTED ? (u64)a.early_row : (u64)a.rows);
  if (SORTED) empty = empty && a.has[row] == 0;
  else empty = empty && (row < a.row_lo || row >= a.row_hi);
  const u64 todo = __ballot(empty);  // the same in every wave
  if (todo == 0) return;
  if (empty && threadIdx.x < 64) rows[__popcll(todo & (((u64)1 << lane) - 1))] = (uint8_t)lane;
  __syncthreads();
  const u32 per_row = a.fill_units.d, units = (u32)__popcll(todo) * per_row;
  for (u32 u = threadIdx.x; u < units; u += kInThreads) {
    const u32 k = quotient(u, a.fill_units);
    zero_unit<GT>(a, a.grad + (int64_t)(r0 + rows[k]) * a.ld_grad, u - k * per_row);
  }
}

// rows of dy in flight per wave
template <bool DROP> constexpr int kSumBatch = DROP ? 4 : 8;

// One wave per (window of a.window places, 512 columns): it sums the chunks that
// begin in the window.  A chunk may end up to its length less one behind it.  The
// workgroups that zero come after those that sum, and keep the memory busy while
// the last of these wait for their rows.
template <class DT, class GT, bool SORTED, bool DROP>
__global__ __launch_bounds__(kInThreads) void grad_sum_kernel(const GradLaunch a) {
  constexpr int W = kWidth<DT, GT>, P = 8 / W, B = kSumBatch<DROP>;
  const u32 group = a.first_group + blockIdx.x;
  if (group >= a.sum_groups) {
    fill_rows<GT, SORTED>(a, (group - a.sum_groups) * a.fill_rows);
    return;
  }
  const u32 lane = threadIdx.x & 63;
  const u32 w = __builtin_amdgcn_readfirstlane(group * (kInThreads / 64) + (threadIdx.x >> 6));
  const u32 win = w / a.slabs, slab = w - win * a.slabs;
  const u32 p0 = win * a.window;
  if (win >= a.windows) return;
  const u32 total = SORTED ? *a.n_valid : a.total;
  uint4 e = make_uint4(0, 0, 0, 0);
  if (p0 + lane < a.places) e = order_at<SORTED>(a, p0 + lane);  // beyond total: not written, not used
  if (p0 >= total) return;

  const u32 chunk = 1u << a.lg_chunk, in_chunk = chunk - 1;
  const u64 heads = __ballot(p0 + lane < total && (e.z & in_chunk) == 0) & (((u64)1 << a.window) - 1);
  if (heads == 0) return;
  const u64 ends = __ballot(p0 + lane < total && ((e.z & in_chunk) == in_chunk || e.z + 1 == e.w));
  const u32 lo = (u32)__builtin_ctzll(heads);
  const u32 last = 63 - (u32)__builtin_clzll(heads);
  const u32 hi = last + (u32)__builtin_ctzll(ends >> last) + 1;  // window + chunk <= 64 places: the end is in sight

  u32 col[P], n[P];
#pragma unroll
  for (int q = 0; q < P; ++q) {
    col[q] = (slab * 64 + piece_group<W>(lane, q)) * kGroup + piece_col<W>(lane);
    n[q] = col[q] < a.dim ? a.dim - col[q] : 0;
  }
  const u32 drop_group = slab * 64 + piece_group<W>(lane, lane & (P - 1));
  const u32 step = DROP ? drop_step(a.drop) : 0;

  float acc[8] = {};
  u32 head = lo;  // of the current chunk
  for (u32 i0 = lo; i0 < hi; i0 += B) {
    Raw<DT, W> x[B][P];
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
      for (int q = 0; q < P; ++q) {
        x[b][q] = Raw<DT, W>{};
        if (i0 + b < hi && n[q]) {
          const u32 t = __builtin_amdgcn_readlane(e.x, i0 + b);
          const u32 d = load_w<DT, W>(a.dy + (int64_t)t * a.ld_dy + (int64_t)col[q] * DT::bytes, a.dy_end, x[b][q]);
          if (a.n - t <= kGroup) move_down<DT, W>(x[b][q], d);
        }
      }
    Words random[B];
    if constexpr (DROP) {
#pragma unroll
      for (int b = 0; b < B; ++b)
        if (i0 + b < hi) random[b] = draw<W>(a.drop, step, __builtin_amdgcn_readlane(e.x, i0 + b), drop_group);
    }
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const u32 i = i0 + b;
      if (i >= hi) break;
      float v[8];
#pragma unroll
      for (int q = 0; q < P; ++q) widen<DT, W>(x[b][q], v + q * W);
      if constexpr (DROP) drop8(a.drop, random[b], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] += v[j];
      if (ends >> i & 1) {
        const u32 len = __builtin_amdgcn_readlane(e.w, i);
        if (len <= chunk) {
          write_row8<GT, W>(a, __builtin_amdgcn_readlane(e.y, i), slab, lane, acc, a.factor);
        } else {
          const bool tail = i + 1 - head < chunk;
          float* const q = a.partial + ((u64)partial_slot(a, p0 + head, tail) * a.slabs + slab) * 512 + lane * 8;
#pragma unroll
          for (int j = 0; j < 8; j += 4)
            *reinterpret_cast<float4*>(q + j) = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
        head = i + 1;
      }
    }
  }
}

// adds the partial rows [j_lo, j_hi) of the run of `len` places that begins at place p
__device__ __forceinline__ void add_partials(const GradLaunch& a, u32 p, u32 len, u32 j_lo, u32 j_hi, u32 slab,
                                             u32 lane, float acc[8]) {
  const u32 full = len >> a.lg_chunk;
#pragma unroll 4
  for (u32 j = j_lo; j < j_hi; ++j) {
    const u32 slot = partial_slot(a, p + (j << a.lg_chunk), j == full);
    const float4* const q = reinterpret_cast<const float4*>(a.partial + ((u64)slot * a.slabs + slab) * 512 + lane * 8);
    const float4 x = q[0], y = q[1];
    acc[0] += x.x; acc[1] += x.y; acc[2] += x.z; acc[3] += x.w;
    acc[4] += y.x; acc[5] += y.y; acc[6] += y.z; acc[7] += y.w;
  }
}

// One workgroup per (a.join_places places, 512 columns).  The runs of several chunks
// that begin there: a wave takes one of few chunks by itself, all waves together
// one of many, each a consecutive part of it.
template <class GT, int W, bool SORTED>
__global__ __launch_bounds__(kJoinThreads) void grad_join_kernel(const GradLaunch a) {
  constexpr u32 NW = kJoinThreads / 64;
  __shared__ uint4 runs[kJoinThreads / kMinChunk];  // (place, row, length, chunks)
  __shared__ u32 n_runs;
  __shared__ float part[NW][64][8];
  const u32 group = a.first_group + blockIdx.x, block = group / a.slabs, slab = group - block * a.slabs;
  const u32 p = block * a.join_places + threadIdx.x, in_chunk = (1u << a.lg_chunk) - 1;
  const u32 total = SORTED ? *a.n_valid : a.total;
  const bool mine = threadIdx.x < a.join_places && p < a.places;
  uint4 e = make_uint4(0, 0, 0, 0);
  if (mine) e = order_at<SORTED>(a, p);
  if (threadIdx.x == 0) n_runs = 0;
  __syncthreads();
  // heads of longer runs are more than a chunk apart
  if (mine && p < total && e.z == 0 && e.w > in_chunk + 1)
    runs[atomicAdd(&n_runs, 1u)] = make_uint4(p, e.y, e.w, (e.w + in_chunk) >> a.lg_chunk);
  __syncthreads();
  const u32 lane = threadIdx.x & 63, wave = threadIdx.x >> 6, count = n_runs;
  for (u32 r = wave; r < count; r += NW) {
    const uint4 run = runs[r];
    if (run.w > NW) continue;
    float acc[8] = {};
    add_partials(a, run.x, run.z, 0, run.w, slab, lane, acc);
    write_row8<GT, W>(a, run.y, slab, lane, acc, a.factor);
  }
  for (u32 r = 0; r < count; ++r) {
    const uint4 run = runs[r];
    if (run.w <= NW) continue;
    const u32 each = (run.w + NW - 1) / NW, lo = min(run.w, wave * each), hi = min(run.w, lo + each);
    float acc[8] = {};
    add_partials(a, run.x, run.z, lo, hi, slab, lane, acc);
#pragma unroll
    for (int j = 0; j < 8; ++j) part[wave][lane][j] = acc[j];
    __syncthreads();
    if (wave == 0) {
      for (u32 w = 1; w < NW; ++w)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += part[w][lane][j];
      write_row8<GT, W>(a, run.y, slab, lane, acc, a.factor);
    }
    __syncthreads();
  }
}

// A small batch in one launch: the workgroup of a class orders its ids in LDS, sums
// its rows and zeroes those without an id.  Waves take (row, 512 columns) each;
// a run of more than kOnceRun ids is summed by all waves together, which still
// leaves a very frequent id to one CU: hence for small batches only.
template <class DT, class GT, bool DROP>
__global__ __launch_bounds__(kSortThreads) void grad_once_kernel(const GradLaunch a) {
  constexpr int W = kWidth<DT, GT>, P = 8 / W, B = 4;
  extern __shared__ u32 lds[];
  __shared__ float part[kSortWaves][64][8];
  const u32 cls = blockIdx.x, *const start = lds + kSortWaves * a.keys, *const tot = start + a.keys;
  u32* const places = lds + (kSortWaves + 2) * a.keys + kSortWaves * a.list;  // [n] the class's positions in order
  const u32 lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  __shared__ u32 first;
  order_class(
      a, cls, lds, [&](u32 before, u32) { if (threadIdx.x == 0) first = before; },
      [&](u32 at, u32 t, u32) { places[at - first] = t; });
  __syncthreads();
  const u32 step = DROP ? drop_step(a.drop) : 0;

  // the sum of the class's places [lo, hi) in a slab
  auto sum = [&](u32 lo, u32 hi, u32 slab, float acc[8]) {
    u32 col[P], n[P];
#pragma unroll
    for (int q = 0; q < P; ++q) {
      col[q] = (slab * 64 + piece_group<W>(lane, q)) * kGroup + piece_col<W>(lane);
      n[q] = col[q] < a.dim ? a.dim - col[q] : 0;
    }
    const u32 drop_group = slab * 64 + piece_group<W>(lane, lane & (P - 1));
    for (u32 i0 = lo; i0 < hi; i0 += B) {
      Raw<DT, W> x[B][P];
      u32 t[B];
#pragma unroll
      for (int b = 0; b < B; ++b) t[b] = __builtin_amdgcn_readfirstlane(places[min(i0 + b, hi - 1)]);
#pragma unroll
      for (int b = 0; b < B; ++b)
#pragma unroll
        for (int q = 0; q < P; ++q) {
          x[b][q] = Raw<DT, W>{};
          if (i0 + b < hi && n[q]) {
            const u32 d = load_w<DT, W>(a.dy + (int64_t)t[b] * a.ld_dy + (int64_t)col[q] * DT::bytes, a.dy_end, x[b][q]);
            if (a.n - t[b] <= kGroup) move_down<DT, W>(x[b][q], d);
          }
        }
      Words random[B];
      if constexpr (DROP) {
#pragma unroll
        for (int b = 0; b < B; ++b)
          if (i0 + b < hi) random[b] = draw<W>(a.drop, step, t[b], drop_group);
      }
#pragma unroll
      for (int b = 0; b < B; ++b) {
        if (i0 + b >= hi) break;
        float v[8];
#pragma unroll
        for (int q = 0; q < P; ++q) widen<DT, W>(x[b][q], v + q * W);
        if constexpr (DROP) drop8(a.drop, random[b], v);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += v[j];
      }
    }
  };

  // long runs first: all waves meet there
  const u32 across = min(a.slabs, (u32)kSortWaves), splits = kSortWaves / across;
  const u32 split = wave / across;
  for (u32 k0 = 0; k0 < a.keys; k0 += 64) {
    u64 longs = __ballot(k0 + lane < a.keys && tot[min(k0 + lane, a.keys - 1)] > kOnceRun);
    for (; longs; longs &= longs - 1) {
      const u32 k = k0 + (u32)__builtin_ctzll(longs), row = (k << a.lg_classes) + cls;
      const u32 len = __builtin_amdgcn_readfirstlane(tot[k]), at = __builtin_amdgcn_readfirstlane(start[k]) - first;
      const u32 each = (len + splits - 1) / splits;
      for (u32 s0 = 0; s0 < a.slabs; s0 += across) {
        const u32 slab = s0 + wave % across;
        float acc[8] = {};
        if (split < splits && slab < a.slabs)
          sum(at + min(len, split * each), at + min(len, (split + 1) * each), slab, acc);
#pragma unroll
        for (int j = 0; j < 8; ++j) part[wave][lane][j] = acc[j];
        __syncthreads();
        if (split == 0 && slab < a.slabs) {
          for (u32 w = 1; w < splits; ++w)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] += part[w * across + wave][lane][j];
          write_row8<GT, W>(a, row, slab, lane, acc, a.factor);
        }
        __syncthreads();
      }
    }
  }
  for (u32 i = wave; i < a.keys * a.slabs; i += kSortWaves) {
    const u32 k = i / a.slabs, slab = i - k * a.slabs;
    const u32 len = __builtin_amdgcn_readfirstlane(tot[k]);
    const u64 row = ((u64)k << a.lg_classes) + cls;
    if (row >= (u64)a.rows || len > kOnceRun || (len == 0 && a.accumulate)) continue;
    float acc[8] = {};
    if (len) {
      const u32 at = __builtin_amdgcn_readfirstlane(start[k]) - first;
      sum(at, at + len, slab, acc);
    }
    write_row8<GT, W>(a, (u32)row, slab, lane, acc, len ? a.factor : 0.0f);  // no id: +0, whatever its sign
  }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

// Units per lane of a lookup: one, or in some forms two from this many units on: bf16
// rows of 4096, 8192 ids (4.2M units) 17.5 us with one against 18.3, 32768 ids (16.8M) 74.7
// against 62.2.  A dropout is never faster with two (8192 x 1600 bf16 with residual
// 13.4 against 13.9 us, 16384 x 4097 fp32 90.9 against 91.8).
constexpr u32 kLookupUnits = 1u << 23;
// The forms (us with one / with two; 42000 x 1600, and 32768 x 4096, where a wave has one
// row; * takes one):
//   16 to 16 bits    35.8 / 31.9, 74.7 / 62.2; with positions 39.8 / 39.9, 90.7 / 83.2;
//                    with dropout 48.9 / 50.3 *, 98.7 / 93.5
//   fp32 to 16 bits  59.7 / 53.9, 89.6 / 91.4 *; with positions 68.5 / 65.2, 114 / 120 *;
//                    with dropout 74.7 / 74.7 *, 119 / 124 *
//   16 bits to fp32  48.6 / 51.2 *, 105 / 106 *; with positions 60.8 / 57.4, 141 / 148 *;
//                    with dropout 70.9 / 72.1 *, 145 / 153 *
//   fp32 to fp32     76.6 / 75.0 *, 122 / 129 *; with positions 92.5 / 99.2 *, 162 / 178 *;
//                    with dropout 96.1 / 96.3 *, 161 / 172 *
template <class TT, class OT, bool DROP, bool ONE>
constexpr bool kTwoUnits = kWidth<TT, OT> == 8 ? ONE || !DROP : !ONE && !DROP && TT::bytes != OT::bytes;
template <class TT, class OT>
bool two_units(const LookupLaunch& a) {
  return a.units >= kLookupUnits && (TT::bytes >= OT::bytes || a.pos_table);
}

// calls f(drop, one row per wave) with constants
template <class F>
void with_form(u32 groups, u32 thr, F&& f) {
  auto one = [&](auto d) { groups % 64 == 0 ? f(d, std::true_type{}) : f(d, std::false_type{}); };
  thr ? one(std::true_type{}) : one(std::false_type{});
}
dim3 stream_grid(u32 units, int per_lane) {
  const u64 per = (u64)kInThreads * per_lane;
  return dim3((u32)((units + per - 1) / per));
}

template <class XT, class OT>
void dropout_as(const DropoutLaunch& a, hipStream_t st) {
  with_form(a.groups.d, a.drop.thr, [&](auto d, auto w) {
    hipLaunchKernelGGL((dropout_kernel<XT, OT, decltype(d)::value, decltype(w)::value>), stream_grid(a.units, 1),
                       dim3(kInThreads), 0, st, a);
  });
}

template <class TT, class OT>
void lookup_as(const LookupLaunch& a, hipStream_t st) {
  with_form(a.groups.d, a.drop.thr, [&](auto d, auto w) {
    constexpr bool DROP = decltype(d)::value, ONE = decltype(w)::value;
    if constexpr (kTwoUnits<TT, OT, DROP, ONE>) {
      if (two_units<TT, OT>(a)) {
        hipLaunchKernelGGL((lookup_kernel<TT, OT, 2, DROP, ONE>), stream_grid(a.units, 2), dim3(kInThreads), 0, st, a);
        return;
      }
    }
    hipLaunchKernelGGL((lookup_kernel<TT, OT, 1, DROP, ONE>), stream_grid(a.units, 1), dim3(kInThreads), 0, st, a);
  });
}

// calls launch(grid) for `groups` workgroups in parts of at most kMaxGroups
template <class F>
void in_parts(GradLaunch& a, u32 groups, F&& launch) {
  for (u64 g = 0; g < groups; g += kMaxGroups) {
    a.first_group = (u32)g;
    launch(dim3((u32)std::min<u64>(groups - g, kMaxGroups)));
  }
}

template <class DT, class GT, bool SORTED>
int grad_as(GradLaunch a, hipStream_t st) {
  const int64_t row_bytes = (int64_t)a.dim * GT::bytes;
  // rows that may begin inside a line have up to a line's worth more units
  a.fill_align = row_bytes < kLineRow ? 1 : 128;
  const bool lines = reinterpret_cast<uintptr_t>(a.grad) % a.fill_align == 0 && a.ld_grad % a.fill_align == 0;
  a.fill_units = fast_div((u32)((row_bytes + (lines ? 0 : a.fill_align - GT::bytes) + 15) / 16));
  if constexpr (SORTED) {
    const u32 range = (a.n + kSortThreads - 1) / kSortThreads * 64;  // positions per wave
    a.list = range < (1u << 22) ? std::min<u32>(range, kSortList) : 0;
    const size_t lds = ((size_t)(kSortWaves + 2) * a.keys + (size_t)kSortWaves * a.list) * sizeof(u32);
    if ((u64)a.n * a.slabs <= kOnceIds && a.rows * row_bytes <= kOnceBytes && a.keys <= kOnceKeys) {
      const dim3 g(1u << a.lg_classes), b(kSortThreads);
      const size_t all = lds + a.n * sizeof(u32);
      if (a.drop.thr) hipLaunchKernelGGL((grad_once_kernel<DT, GT, true>), g, b, all, st, a);
      else hipLaunchKernelGGL((grad_once_kernel<DT, GT, false>), g, b, all, st, a);
      return launched("embedding gradient");
    }
    u32 early_groups = 0;
    a.early_row = (u32)a.rows;
    if (!a.accumulate) {
      // as many as fit beside the sort, 64 KiB or one row a workgroup
      a.early_rows = (u32)std::max<int64_t>(1, kEarlyGroupBytes / row_bytes);
      const int64_t bytes = kEarlyBytes + kEarlyBytesPerId * (int64_t)a.n;
      // (there are at most 2 kMaxGroups classes, so that the launch has fewer than 2^32 threads)
      early_groups = (u32)std::min<int64_t>(std::min<int64_t>(a.rows, bytes / row_bytes) / a.early_rows, kMaxGroups);
      a.early_row = (u32)(a.rows - (int64_t)early_groups * a.early_rows);
    }
    hipLaunchKernelGGL(sort_kernel<GT>, dim3((1u << a.lg_classes) + early_groups), dim3(kSortThreads), lds, st, a);
    if (int rc = launched("embedding gradient (order)")) return rc;
  }
  const u64 waves = (u64)a.windows * a.slabs;
  a.sum_groups = (u32)((waves + 3) / 4);
  a.fill_rows = (u32)std::max<int64_t>(1, std::min<int64_t>(64, kFillBytes / row_bytes));
  const bool fill = !a.accumulate && (SORTED || a.rows > (int64_t)(a.row_hi - a.row_lo));
  const int64_t fill_to = SORTED ? (int64_t)a.early_row : a.rows;
  const u32 fill_groups = fill ? (u32)((fill_to + a.fill_rows - 1) / a.fill_rows) : 0;
  if (a.sum_groups + fill_groups == 0) return ZERO_OK;
  in_parts(a, a.sum_groups + fill_groups, [&](dim3 g) {
    if (a.drop.thr) hipLaunchKernelGGL((grad_sum_kernel<DT, GT, SORTED, true>), g, dim3(kInThreads), 0, st, a);
    else hipLaunchKernelGGL((grad_sum_kernel<DT, GT, SORTED, false>), g, dim3(kInThreads), 0, st, a);
  });
  if (int rc = launched("embedding gradient (sums)")) return rc;
  if (a.places > 0 && a.longest > 1u << a.lg_chunk) {
    // few places leave each workgroup few runs, many of them keep the workgroups few
    a.join_places = kJoinThreads;
    while (a.join_places > 64 && (u64)a.places * a.slabs < (u64)a.join_places * kJoinGroups) a.join_places /= 2;
    const u32 blocks = (a.places + a.join_places - 1) / a.join_places;
    in_parts(a, blocks * a.slabs, [&](dim3 g) {
      hipLaunchKernelGGL((grad_join_kernel<GT, kWidth<DT, GT>, SORTED>), g, dim3(kJoinThreads), 0, st, a);
    });
  }
  return launched("embedding gradient (joins)");
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

// Chunks of a run: long ones need fewer partial rows, short ones spread a small
// batch over more waves.
uint32_t grad_lg_chunk(int64_t n_ids, int64_t dim) {
  const int64_t slabs = (dim + 511) / 512;
  uint32_t lg = kMaxLgChunk;
  while ((1u << lg) > kMinChunk && (n_ids >> (lg - 1)) * slabs < kGradWaves) --lg;
  return lg;
}

int launch_dropout(const DropoutLaunch& a, zero_dtype_t xt, zero_dtype_t ot, void* stream) {
  if (a.x_end - a.x < kGroup * (xt == ZERO_F32 ? 4 : 2) || (a.res && a.res_end - a.res < kGroup * (ot == ZERO_F32 ? 4 : 2))) {
    hipLaunchKernelGGL(dropout_short_kernel, dim3(1), dim3(64), 0, (hipStream_t)stream, a, (int)xt, (int)ot);
    return launched("dropout");
  }
  return with_types(xt, ot, [&](auto x, auto o) {
    dropout_as<decltype(x), decltype(o)>(a, (hipStream_t)stream);
    return launched("dropout");
  });
}

int launch_lookup(const LookupLaunch& a, zero_dtype_t tt, zero_dtype_t ot, void* stream) {
  const int64_t least = kGroup * (tt == ZERO_F32 ? 4 : 2);
  if ((a.rows > 0 && a.table_end - a.table < least) || (a.pos_table && a.pos_rows > 0 && a.pos_end - a.pos_table < least)) {
    const u64 blocks = std::min<u64>(((u64)a.n * a.dim + 255) / 256, kMaxGroups);
    hipLaunchKernelGGL(lookup_short_kernel, dim3((u32)blocks), dim3(256), 0, (hipStream_t)stream, a, (int)tt, (int)ot);
    return launched("embedding lookup");
  }
  return with_types(tt, ot, [&](auto t, auto o) {
    lookup_as<decltype(t), decltype(o)>(a, (hipStream_t)stream);
    return launched("embedding lookup");
  });
}

int launch_embed_grad(const GradLaunch& a, zero_dtype_t dt, zero_dtype_t gt, void* stream) {
  if (a.n > 0 && a.dy_end - a.dy < kGroup * (dt == ZERO_F32 ? 4 : 2)) {
    const u64 blocks = std::min<u64>(((u64)a.rows * a.dim + 255) / 256, kMaxGroups);
    hipLaunchKernelGGL(grad_short_kernel, dim3((u32)blocks), dim3(256), 0, (hipStream_t)stream, a, (int)dt, (int)gt);
    return launched("embedding gradient");
  }
  return with_types(dt, gt, [&](auto d, auto g) {
    if (a.ids) return grad_as<decltype(d), decltype(g), true>(a, (hipStream_t)stream);
    return grad_as<decltype(d), decltype(g), false>(a, (hipStream_t)stream);
  });
}

}  // namespace zk
