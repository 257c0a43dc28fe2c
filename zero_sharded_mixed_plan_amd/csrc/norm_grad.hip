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

template <class AT, class ST, bool HELD, int C>
struct GradRow {
  Raw8<AT> dy[C];
  Raw8<ST> h[HELD ? 1 : C], dres[C];
  RawHeld q[HELD ? C : 1];
  float rstd;
};

template <class AT, class ST, bool HELD, int WAVES, int C>
__device__ __forceinline__ void load_row(const RmsGradLaunch& a, int64_t row, u32 t, const u32 (&n)[C],
                                         GradRow<AT, ST, HELD, C>& r) {
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const u32 grp = c * WAVES * 64 + t;
    load8<AT>(a.dy + row * a.ld_dy + (int64_t)grp * 8 * AT::bytes, a.dy_end, n[c], r.dy[c]);
    if constexpr (HELD) load_held(a.held, row, grp, n[c], r.q[c]);
    else load8<ST>(a.h + row * a.ld_h + (int64_t)grp * 8 * ST::bytes, a.h_end, n[c], r.h[c]);
    if (a.dres) load8<ST>(a.dres + row * a.ld_dres + (int64_t)grp * 8 * ST::bytes, a.dres_end, n[c], r.dres[c]);
  }
  r.rstd = a.rstd[row];
}

template <class AT, class ST, bool HELD, int WAVES, int C>
__global__ __launch_bounds__(grad_threads(WAVES)) void rms_grad_kernel(const RmsGradLaunch a) {
  constexpr u32 kRow = WAVES * 64;
  constexpr u32 kRows = grad_threads(WAVES) / kRow;  // rows at a time
  __shared__ float part[2][WAVES];
  __shared__ float joined[kRows > 1 ? kRows - 1 : 1][kRows > 1 ? kRow * C * 8 : 1];
  const u32 t = threadIdx.x % kRow, mine = threadIdx.x / kRow;
  u32 n[C];
  float w[C][8], sum[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const u32 col = (c * kRow + t) * 8;
    n[c] = col < a.cols ? min(a.cols - col, 8u) : 0;
    Raw8<F32> q;
    if (a.weight) {
      load8_as(a.weight + (int64_t)col * one_bytes(a.weight_type), a.weight_end, a.weight_type, n[c], q);
      values8_as(q, a.weight_type, n[c], w[c]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (!a.weight) w[c][j] = 1.0f;
      sum[c][j] = 0.0f;
    }
  }
  const int64_t stride = (int64_t)gridDim.x * kRows;
  int64_t row = (int64_t)blockIdx.x * kRows + mine;
  GradRow<AT, ST, HELD, C> next;
  if (row < a.rows) load_row<AT, ST, HELD, WAVES, C>(a, row, t, n, next);
  for (u32 turn = 0; row < a.rows; row += stride, ++turn) {
#pragma unroll
    for (int c = 0; c < C; ++c) asm volatile("" : "+v"(n[c]));  // no lane masks of it are kept across rows
    const GradRow<AT, ST, HELD, C> r = next;
    if (row + stride < a.rows) load_row<AT, ST, HELD, WAVES, C>(a, row + stride, t, n, next);
    float dot = 0.0f, v[C][8], s[C][8];  // v: n
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
    dot = wave_sum(dot);
    if constexpr (WAVES > 1) {
      if (t % 64 == 0) part[turn & 1][t / 64] = dot;
      __syncthreads();
      dot = 0.0f;
#pragma unroll
      for (int i = 0; i < WAVES; ++i) dot += part[turn & 1][i];
    }
    dot /= (float)a.cols;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float d[8];
      if (a.dres) values8<ST>(r.dres[c], n[c], d);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float g = r.rstd * __builtin_fmaf(-v[c][j], dot, s[c][j]);
        d[j] = a.dres ? g + d[j] : g;
      }
      store8<ST>(a.dh + row * a.ld_dh + (int64_t)(c * kRow + t) * 8 * ST::bytes, d, n[c]);
    }
  }
  if (!a.dweight) return;
  if constexpr (kRows > 1) {
    if (mine > 0) {
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) joined[mine - 1][(c * kRow + t) * 8 + j] = sum[c][j];
    }
    __syncthreads();
    if (mine > 0) return;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (u32 i = 0; i + 1 < kRows; ++i) sum[c][j] += joined[i][(c * kRow + t) * 8 + j];
  }
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (u32 j = 0; j < 8; ++j)
      if (j < n[c]) a.partial[(int64_t)blockIdx.x * a.cols + (c * kRow + t) * 8 + j] = sum[c][j];
}

// 32 columns a workgroup, 32 slices of the partial rows
constexpr int kJoinCols = 32, kJoinSlices = 32;
__global__ __launch_bounds__(kJoinCols * kJoinSlices) void rms_grad_join_kernel(const RmsGradLaunch a) {
  __shared__ double part[kJoinSlices][kJoinCols];
  const u32 x = threadIdx.x % kJoinCols, slice = threadIdx.x / kJoinCols;
  const u32 col = blockIdx.x * kJoinCols + x;
  double sum = 0.0;
  if (col < a.cols)
    for (u32 p = slice; p < a.partials; p += kJoinSlices) sum += (double)a.partial[(int64_t)p * a.cols + col];
  part[slice][x] = sum;
  __syncthreads();
  if (slice != 0 || col >= a.cols) return;
  sum = 0.0;
  for (int i = 0; i < kJoinSlices; ++i) sum += part[i][x];
  char* const p = a.dweight + (int64_t)col * one_bytes(a.dweight_type);
  if (a.accumulate) sum += (double)load_one(p, a.dweight_type);
  store_one(p, a.dweight_type, (float)sum);
}

int rows_at_a_time(int64_t cols) { return cols <= 1024 ? 4 : 1; }

template <class AT, class ST, bool HELD>
void grad_as(const RmsGradLaunch& a, hipStream_t s) {
  auto go = [&](auto waves, auto groups) {
    constexpr int W = decltype(waves)::value, C = decltype(groups)::value;
    hipLaunchKernelGGL((rms_grad_kernel<AT, ST, HELD, W, C>), dim3(a.partials), dim3(grad_threads(W)), 0, s, a);
  };
#define ZK_SHAPE(w, c) go(std::integral_constant<int, w>{}, std::integral_constant<int, c>{})
  if (a.cols <= 512) ZK_SHAPE(1, 1);
  else if (a.cols <= 1024) ZK_SHAPE(1, 2);
  else if (a.cols <= 2048) ZK_SHAPE(4, 1);
  else if (a.cols <= 4096) ZK_SHAPE(4, 2);
  else ZK_SHAPE(8, 2);
#undef ZK_SHAPE
}

}  // namespace

// Workgroups that go through the rows, as many as fit the card at once.
uint32_t rms_grad_partials(int64_t rows, int64_t cols) {
  const int64_t at_once = rows_at_a_time(cols);
  return (uint32_t)std::max<int64_t>(1, std::min<int64_t>((rows + at_once - 1) / at_once, cols <= 4096 ? 1024 : 512));
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
