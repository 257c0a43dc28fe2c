// HIP kernels for gfx950 (CDNA4): the gradient of RMS norm.
//
// With n = h * rstd and s = weight * dy:
//   dh = rstd * (s - n * mean(s * n)) + the residual path's gradient
//   dweight = sum over the rows of dy * n
//
// Bound by HBM.  A workgroup goes through many rows, so that the weight's gradient is summed
// in registers; each workgroup leaves one row of partial sums, and a second launch adds
// those in fp64, in an order that the sizes alone give.  The next row's values load
// while a row is summed.
#include <algorithm>

#include "held.h"

namespace zk {
namespace {

constexpr int grad_threads(int waves) { return waves < 4 ? 256 : waves * 64; }

// A row is WAVES waves of C times 8 columns a lane; short rows share a workgroup of four waves.
template <class AT, class ST, bool HELD, int WAVES, int C>
__global__ __launch_bounds__(grad_threads(WAVES)) void rms_grad_kernel(const RmsGradLaunch a) {
  constexpr u32 kRow = WAVES * 64;
  constexpr u32 kRows = grad_threads(WAVES) / kRow;  // rows at a time
  __shared__ float part[2][kRows][WAVES];            // two, for a wave may be a row ahead
  __shared__ float joined[kRows > 1 ? kRows - 1 : 1][kRows > 1 ? C * kRow * 8 : 1];
  // a wave's row is a number of the wave, so that its addresses cost no vector instructions
  const u32 t = kRows == 1 ? threadIdx.x : threadIdx.x % kRow;
  const u32 mine = kRows == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / kRow);
  u32 n[C];
  float w[C][8], sum[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const u32 col = (c * kRow + t) * 8;
    n[c] = col < a.cols ? min(a.cols - col, 8u) : 0;
    if (a.weight) {
      Raw8<F32> rw;
      load8_as(a.weight + (int64_t)col * one_bytes(a.weight_type), a.weight_end, a.weight_type, n[c], rw);
      values8_as(rw, a.weight_type, n[c], w[c]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (!a.weight) w[c][j] = 1.0f;
      sum[c][j] = 0.0f;
    }
  }
  const int64_t stride = (int64_t)gridDim.x * kRows;
  struct Row {
    Raw8<AT> dy[C];
    Raw8<ST> h[HELD ? 1 : C], dres[C];
    RawHeld q[HELD ? C : 1];
    float rstd;
  } next;
  auto load = [&](int64_t row) {
    if (row >= a.rows) return;
    const bool inside = row + 1 < a.rows && a.cols >= 8;  // what follows a row is the next one
    const char* const dy = a.dy + row * a.ld_dy;
    const char* const h = a.h + row * a.ld_h;
    const char* const dres = a.dres + row * a.ld_dres;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const u32 grp = c * kRow + t;
      load8<AT>(dy + grp * 8 * AT::bytes, a.dy_end, n[c], next.dy[c], inside);
      if constexpr (HELD) load_held(a.held, row, grp, n[c], next.q[c], inside);
      else load8<ST>(h + grp * 8 * ST::bytes, a.h_end, n[c], next.h[c], inside);
      if (a.dres) load8<ST>(dres + grp * 8 * ST::bytes, a.dres_end, n[c], next.dres[c], inside);
    }
    next.rstd = a.rstd[row];
  };
  load((int64_t)blockIdx.x * kRows + mine);
  u32 turn = 0;
  // of several rows at a time, all go through the loop as often, for they meet at the barrier
  for (int64_t row0 = (int64_t)blockIdx.x * kRows; row0 < a.rows; row0 += stride, ++turn) {
#pragma unroll
    for (int c = 0; c < C; ++c) asm volatile("" : "+v"(n[c]));  // no lane masks of it are kept across rows
    const int64_t row = row0 + mine;
    const bool exists = kRows == 1 || row < a.rows;
    const Row r = next;
    load(row + stride);
    float dot = 0.0f, v[C][8], s[C][8];  // v: n
    if (exists) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if constexpr (HELD) held_values(r.q[c], n[c], v[c]);
        else values8<ST>(r.h[c], n[c], v[c]);
        values8<AT>(r.dy[c], n[c], s[c]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[c][j] *= r.rstd;
          sum[c][j] = __builtin_fmaf(s[c][j], v[c][j], sum[c][j]);
          s[c][j] *= w[c][j];
          dot = __builtin_fmaf(s[c][j], v[c][j], dot);
        }
      }
    }
    dot = wave_sum(dot);
    if constexpr (WAVES > 1) {
      if (t % 64 == 0) part[turn & 1][mine][t / 64] = dot;
      __syncthreads();
      dot = 0.0f;
#pragma unroll
      for (int i = 0; i < WAVES; ++i) dot += part[turn & 1][mine][i];
    }
    if (!exists) continue;
    dot /= (float)a.cols;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float d[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) s[c][j] = r.rstd * __builtin_fmaf(-v[c][j], dot, s[c][j]);
      if (a.dres) {
        values8<ST>(r.dres[c], n[c], d);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[c][j] += d[j];
      }
      store8<ST>(a.dh + row * a.ld_dh + (c * kRow + t) * 8 * ST::bytes, s[c], n[c]);
    }
  }
  if (!a.dweight) return;
  if constexpr (kRows > 1) {
    if (mine > 0) {
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) joined[mine - 1][(c * 8 + j) * kRow + t] = sum[c][j];
    }
    __syncthreads();
    if (mine > 0) return;
#pragma unroll
    for (u32 i = 0; i + 1 < kRows; ++i)
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[c][j] += joined[i][(c * 8 + j) * kRow + t];
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const u32 col = (c * kRow + t) * 8;
    store8<F32>(reinterpret_cast<char*>(a.partial + (int64_t)blockIdx.x * a.cols + col), sum[c], n[c]);
  }
}

// A sum in fp32 that a second rounding, to 16 bits, takes where one rounding of the sum itself would: what fp32
// cuts off makes its last bit odd, so that no sum lands on the middle of two 16-bit numbers that was not there.
__device__ __forceinline__ float to_odd(double v) {
  const float f = (float)v;
  const double d = (double)f;
  if (d == v || v != v) return f;
  return __uint_as_float((__float_as_uint(f) - (fabs(d) > fabs(v) ? 1 : 0)) | 1);
}

// 32 columns a workgroup, 32 slices of the partial rows
constexpr int kJoinCols = 32, kJoinSlices = 32;
__global__ __launch_bounds__(kJoinCols * kJoinSlices) void rms_grad_join_kernel(const RmsGradLaunch a) {
  __shared__ double part[kJoinSlices][kJoinCols];
  const u32 x = threadIdx.x % kJoinCols, slice = threadIdx.x / kJoinCols;
  const u32 col = blockIdx.x * kJoinCols + x;
  double sum = 0.0;
  if (col < a.cols) {
#pragma unroll 4
    for (u32 p = slice; p < a.partials; p += kJoinSlices) sum += (double)a.partial[(int64_t)p * a.cols + col];
  }
  part[slice][x] = sum;
  __syncthreads();
  if (slice != 0 || col >= a.cols) return;
  sum = 0.0;
  for (int i = 0; i < kJoinSlices; ++i) sum += part[i][x];
  char* const p = a.dweight + (int64_t)col * one_bytes(a.dweight_type);
  if (a.accumulate) sum += (double)load_one(p, a.dweight_type);
  store_one(p, a.dweight_type, a.dweight_type == ZERO_F32 ? (float)sum : to_odd(sum));
}

// 8 columns a lane: with 16, 8192 x 4096 bf16 took 40.5 us from 8 bits, against 37.6, and 45.1 from tensors, against 43.6.
int waves_of(int64_t cols) { return cols <= 512 ? 1 : cols <= 1024 ? 2 : cols <= 2048 ? 4 : cols <= 4096 ? 8 : 16; }

template <class AT, class ST, bool HELD>
void grad_as(const RmsGradLaunch& a, hipStream_t s) {
  auto go = [&](auto waves) {
    constexpr int W = decltype(waves)::value;
    hipLaunchKernelGGL((rms_grad_kernel<AT, ST, HELD, W, 1>), dim3(a.partials), dim3(grad_threads(W)), 0, s, a);
  };
  switch (waves_of(a.cols)) {
    case 1: return go(std::integral_constant<int, 1>{});
    case 2: return go(std::integral_constant<int, 2>{});
    case 4: return go(std::integral_constant<int, 4>{});
    case 8: return go(std::integral_constant<int, 8>{});
    default: return go(std::integral_constant<int, 16>{});
  }
}

}  // namespace

// Workgroups that go through the rows: as many as fit the card at once, or fewer where each would have
// fewer than four turns, but one a CU.
uint32_t rms_grad_partials(int64_t rows, int64_t cols) {
  const int waves = waves_of(cols), at_once = waves < 4 ? 4 / waves : 1;
  const int64_t groups = (rows + at_once - 1) / at_once, fit = 256 * 16 / std::max(waves, 4);
  return (uint32_t)std::max<int64_t>(1, std::min(groups, std::min(fit, std::max<int64_t>(256, groups / 4))));
}

int64_t rms_grad_partials_most(int64_t rows) { return std::max<int64_t>(1, std::min<int64_t>(rows, 1024)); }

int launch_rms_grad(const RmsGradLaunch& a, zero_dtype_t at, zero_dtype_t st, void* stream) {
  auto run = [&](auto x, auto y) -> int {
    using A = decltype(x);
    using S = decltype(y);
    if (a.rows > 0) {
      if (a.held.codes) grad_as<A, S, true>(a, (hipStream_t)stream);
      else grad_as<A, S, false>(a, (hipStream_t)stream);
      if (int rc = launched("RMS norm gradient")) return rc;
    }
    if (!a.dweight) return ZERO_OK;
    hipLaunchKernelGGL(rms_grad_join_kernel, dim3((a.cols + kJoinCols - 1) / kJoinCols), dim3(kJoinCols * kJoinSlices), 0,
                       (hipStream_t)stream, a);
    return launched("RMS norm gradient (weight)");
  };
  if (at == st) return at == ZERO_F32 ? run(F32{}, F32{}) : at == ZERO_BF16 ? run(BF16{}, BF16{}) : run(F16{}, F16{});
  return at == ZERO_BF16 ? run(BF16{}, F32{}) : run(F16{}, F32{});
}

}  // namespace zk
