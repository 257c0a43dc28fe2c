// HIP kernels for gfx950 (CDNA4): RMS norm of a residual stream.
//
//   h = x + residual, rounded to the stream's type
//   rstd = 1 / sqrt(mean(h^2) + eps)
//   y = h * rstd * weight
//
// Bound by HBM: each element is read once and written once, a row's values wait in
// registers for the row's sum.  The sum and y are computed in fp64, which on this
// card costs a vector instruction no more than fp32 does: the 8-bit codes, where a last bit decides
// which of two values 2^-4 apart is stored, then do not hang on the order of a
// row's sum, and so not on how a row is split over lanes and waves.
#include <algorithm>

#include "held.h"

namespace zk {
namespace {

// A row is WAVES waves of C groups of 8 columns a lane.  Rows of one wave share a
// workgroup of four, so that a workgroup's four waves never wait for each other there.
constexpr int rms_threads(int waves) { return waves < 4 ? 256 : waves * 64; }

template <class XT, class RT, int WAVES, int C, bool HELD>
__global__ __launch_bounds__(rms_threads(WAVES)) void rms_kernel(const RmsLaunch a) {
  constexpr u32 kRow = WAVES * 64;
  constexpr u32 kRows = rms_threads(WAVES) / kRow;
  const u32 t = threadIdx.x % kRow;
  for (int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / kRow; row < a.rows; row += (int64_t)gridDim.x * kRows) {
    Raw8<XT> x[C];
    Raw8<RT> r[C];
    u32 n[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const u32 col = (c * kRow + t) * 8;
      n[c] = col < a.cols ? min(a.cols - col, 8u) : 0;
      asm volatile("" : "+v"(n[c]));  // no lane masks of it are kept across rows, in scalar registers
      load8<XT>(a.x + row * a.ld_x + (int64_t)col * XT::bytes, a.x_end, n[c], x[c]);
    }
    if (a.res) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const u32 col = (c * kRow + t) * 8;
        load8<RT>(a.res + row * a.ld_res + (int64_t)col * RT::bytes, a.res_end, n[c], r[c]);
      }
    }
    float h[C][8];
    double sum = 0.0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      values8<XT>(x[c], n[c], h[c]);
      if (a.res) {
        float q[8];
        values8<RT>(r[c], n[c], q);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const u32 b = bits_of<RT>(h[c][j] + q[j]);
          if constexpr (RT::bytes == 4) h[c][j] = __uint_as_float(b);
          else if constexpr (std::is_same<RT, BF16>::value) h[c][j] = __uint_as_float(b << 16);
          else h[c][j] = (float)__builtin_bit_cast(_Float16, (uint16_t)b);
        }
        const u32 col = (c * kRow + t) * 8;
        store8<RT>(a.total + row * a.ld_total + (int64_t)col * RT::bytes, h[c], n[c]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = __builtin_fma((double)h[c][j], (double)h[c][j], sum);
    }
    sum = wave_sum(sum);
    if constexpr (WAVES > 1) {
      __shared__ double part[2][WAVES];  // two, for a wave may be a row ahead
      const u32 which = (u32)((row / gridDim.x) & 1);
      if (t % 64 == 0) part[which][t / 64] = sum;
      __syncthreads();
      sum = 0.0;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) sum += part[which][w];
    }
#pragma unroll
    for (int c = 0; c < C; ++c) asm volatile("" : "+v"(n[c]));
    const double rstd = 1.0 / __builtin_sqrt(sum / a.cols + a.eps);
    if (a.rstd && t == 0) a.rstd[row] = (float)rstd;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const u32 col = (c * kRow + t) * 8;
      float y[8], w[8];
      if (a.weight) {
        Raw8<F32> q;
        load8_as(a.weight + (int64_t)col * one_bytes(a.weight_type), a.weight_end, a.weight_type, n[c], q);
        values8_as(q, a.weight_type, n[c], w);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double v = (double)h[c][j] * rstd;
        y[j] = (float)(a.weight ? v * (double)w[j] : v);
      }
      clear_tail(y, n[c]);  // infinity times the zeros there
      if (a.y) store8_as(a.y + row * a.ld_y + (int64_t)col * one_bytes(a.y_type), a.y_type, y, n[c]);
      if constexpr (HELD) hold8(a.held, row, c * kRow + t, y, n[c]);
    }
  }
}

template <class XT, class RT, bool HELD>
void rms_as(const RmsLaunch& a, hipStream_t s) {
  auto go = [&](auto waves, auto groups) {
    constexpr int W = decltype(waves)::value, C = decltype(groups)::value;
    constexpr int rows = rms_threads(W) / (W * 64);
    const u32 grid = (u32)std::min<int64_t>((a.rows + rows - 1) / rows, kMaxGroups);
    hipLaunchKernelGGL((rms_kernel<XT, RT, W, C, HELD>), dim3(grid), dim3(rms_threads(W)), 0, s, a);
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

int launch_rms(const RmsLaunch& a, zero_dtype_t xt, zero_dtype_t rt, void* stream) {
  auto run = [&](auto x, auto r) {
    using X = decltype(x);
    using R = decltype(r);
    if (a.held.codes) rms_as<X, R, true>(a, (hipStream_t)stream);
    else rms_as<X, R, false>(a, (hipStream_t)stream);
    return launched("RMS norm");
  };
  if (xt == rt) return xt == ZERO_F32 ? run(F32{}, F32{}) : xt == ZERO_BF16 ? run(BF16{}, BF16{}) : run(F16{}, F16{});
  return xt == ZERO_BF16 ? run(BF16{}, F32{}) : run(F16{}, F32{});  // 16-bit results onto an fp32 stream
}

}  // namespace zk
