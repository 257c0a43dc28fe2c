// HIP kernels for gfx950 (CDNA4): RMS norm of a residual stream.
//
//   h = x + residual, rounded to the stream's type
//   rstd = 1 / sqrt(mean(h^2) + eps)
//   y = h * rstd * weight
//
// Bound by HBM: each element is read once and written once, a row's values wait in
// registers for the row's sum.  In 8-bit codes a last bit decides which of two values 2^-4 apart is
// stored, so rstd and y must not hang on how a row is split over lanes and waves: squares are summed in
// fp64, and y is computed in pairs of fp32 numbers (good to 2^-44), rounded once to
// fp32.  8192 x 4096 bf16, three sets of matrices in turn without a pause: with a residual 51 us, without 26 (53 and
// 28 call by call); all in fp64, whose conversions are slow, 36 without.
#include <algorithm>

#include "held.h"

namespace zk {
namespace {

// A row is WAVES waves of C times 8 columns a lane.  Short rows share a workgroup of four waves.  128 registers,
// four waves a SIMD: the compiler takes 129 to 134 else in wide forms with 8-bit results or an fp32 stream, which
// leaves three (8192 x 8192 bf16 with a residual and 8-bit results 123 us in place of 111, 8192 x 6000 103 and 88).
constexpr int rms_threads(int waves) { return waves < 4 ? 256 : waves * 64; }

// 1 / sqrt(x): the hardware's estimate and two of Newton's steps, each of which squares its error;
// infinity for 0, 0 for infinity.
__device__ __forceinline__ double inverse_root(double x) {
  const double first = __builtin_amdgcn_rsq(x), half = -0.5 * x;
  double r = first;
#pragma unroll
  for (int i = 0; i < 2; ++i) r = __builtin_fma(r * 0.5, __builtin_fma(half * r, r + r, 1.0), r);
  return x == 0.0 || first == 0.0 ? first : r;
}

template <class XT, class RT, int WAVES, int C, bool HELD>
__global__ __launch_bounds__(rms_threads(WAVES), 4) void rms_kernel(const RmsLaunch a) {
  constexpr u32 kRow = WAVES * 64;
  constexpr u32 kRows = rms_threads(WAVES) / kRow;
  // a wave's row is a number of the wave, so that its addresses cost no vector instructions
  const u32 t = kRows == 1 ? threadIdx.x : threadIdx.x % kRow;
  const u32 mine = kRows == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / kRow);
  u32 n[C];
  Raw8<F32> rw[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const u32 col = (c * kRow + t) * 8;
    n[c] = col < a.cols ? min(a.cols - col, 8u) : 0;
    if (a.weight) load8_as(a.weight + (int64_t)col * one_bytes(a.weight_type), a.weight_end, a.weight_type, n[c], rw[c]);
  }
  const int64_t stride = (int64_t)gridDim.x * kRows;
  struct Row {
    Raw8<XT> x[C];
    Raw8<RT> r[C];
  } next;
  auto load = [&](int64_t row) {
    if (row >= a.rows) return;
    const bool inside = row + 1 < a.rows && a.cols >= 8;  // what follows a row is the next one
    const char* const x = a.x + row * a.ld_x;
    const char* const r = a.res + row * a.ld_res;
#pragma unroll
    for (int c = 0; c < C; ++c) load8<XT>(x + (c * kRow + t) * 8 * XT::bytes, a.x_end, n[c], next.x[c], inside);
    if (!a.res) return;
#pragma unroll
    for (int c = 0; c < C; ++c) load8<RT>(r + (c * kRow + t) * 8 * RT::bytes, a.res_end, n[c], next.r[c], inside);
  };
  load((int64_t)blockIdx.x * kRows + mine);
  u32 turn = 0;
  // of several rows at a time, all go through the loop as often, for they meet at the barrier
  for (int64_t row0 = (int64_t)blockIdx.x * kRows; row0 < a.rows; row0 += stride, ++turn) {
#pragma unroll
    for (int c = 0; c < C; ++c) asm volatile("" : "+v"(n[c]));  // no lane masks of it are kept across rows, in scalar registers
    const int64_t row = row0 + mine;
    const bool exists = kRows == 1 || row < a.rows;
    const Row now = next;
    load(row + stride);
    float h[C][8];
    double sum = 0.0;
    if (exists) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        values8<XT>(now.x[c], n[c], h[c]);
        if (a.res) {
          float q[8];
          values8<RT>(now.r[c], n[c], q);
#pragma unroll
          for (int j = 0; j < 8; ++j) h[c][j] += q[j];
          const Raw8<RT> total = round8<RT>(h[c]);
          store8<RT>(a.total + row * a.ld_total + (c * kRow + t) * 8 * RT::bytes, total, n[c]);
          values8<RT>(total, 8, h[c]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = __builtin_fma((double)h[c][j], (double)h[c][j], sum);
      }
    }
    sum = wave_sum(sum);
    if constexpr (WAVES > 1) {
      __shared__ double part[2][kRows][WAVES];  // two, for a wave may be a row ahead
      const u32 which = turn & 1;
      if (t % 64 == 0) part[which][mine][t / 64] = sum;
      __syncthreads();
      sum = 0.0;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) sum += part[which][mine][w];
    }
    if (!exists) continue;
    const RmsLaunch& b = argument<RmsLaunch>();
    const double rstd = inverse_root(sum * b.per_col + b.eps);
    if (b.rstd && t == 0) b.rstd[row] = (float)rstd;
    // The row is scaled by rstd's power of two first, exactly, so that neither an rstd near the ends of
    // fp32 nor its second part is lost: n = h * rstd is of size one.
    const int e = __builtin_amdgcn_frexp_exp(rstd);
    const double m = __builtin_amdgcn_frexp_mant(rstd);
    const float m_hi = (float)m, m_lo = (float)(m - (double)m_hi);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float y[8];
      if (a.weight) {
        float w[8];
        values8_as(rw[c], a.weight_type, 8, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float s = __builtin_amdgcn_ldexpf(h[c][j], e);
          const float p = s * m_hi;
          const float p_lo = __builtin_fmaf(s, m_lo, __builtin_fmaf(s, m_hi, -p));
          // bounded, or an infinite weight times a second part of 0, or of the other sign, would not be a number
          const float q_lo = __builtin_amdgcn_fmed3f(w[j] * p_lo, -0x1.fffffep127f, 0x1.fffffep127f);
          y[j] = __builtin_fmaf(w[j], p, q_lo);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float s = __builtin_amdgcn_ldexpf(h[c][j], e);
          y[j] = __builtin_fmaf(s, m_hi, s * m_lo);
        }
      }
      clear_tail(y, n[c]);  // infinity times the zeros there
      if (b.y) store8_as(b.y + row * b.ld_y + (int64_t)((c * kRow + t) * 8) * one_bytes(b.y_type), b.y_type, y, n[c]);
      if constexpr (HELD) hold8(b.held, row, c * kRow + t, y, n[c]);
    }
  }
}

template <class XT, class RT, bool HELD>
void rms_as(const RmsLaunch& a, hipStream_t s) {
  auto go = [&](auto waves, auto groups) {
    constexpr int W = decltype(waves)::value, C = decltype(groups)::value, rows = rms_threads(W) / (W * 64);
    // as many workgroups as fit the card at once; each loads its next row while it works on one
    const u32 grid = (u32)std::min<int64_t>((a.rows + rows - 1) / rows, 256 * 16 / std::max(W, 4));
    hipLaunchKernelGGL((rms_kernel<XT, RT, W, C, HELD>), dim3(grid), dim3(rms_threads(W)), 0, s, a);
  };
  // 16 bytes of a row a lane and vector: two groups of 16-bit columns (8192 x 4096 bf16 without a residual 26 us,
  // with one 30; 8192 x 8192 53 and 77; slower only onto an fp32 stream with 8-bit results, 8192 x 4096 94 and
  // 83), one of fp32 (4096 x 4096 26 us; with two a form spills)
  constexpr int C = XT::bytes == 4 ? 1 : 2;
  using Groups = std::integral_constant<int, C>;
  if (a.cols <= 512) go(std::integral_constant<int, 1>{}, std::integral_constant<int, 1>{});
  else if (a.cols <= 1024) go(std::integral_constant<int, 2 / C>{}, Groups{});
  else if (a.cols <= 2048) go(std::integral_constant<int, 4 / C>{}, Groups{});
  else if (a.cols <= 4096) go(std::integral_constant<int, 8 / C>{}, Groups{});
  else go(std::integral_constant<int, 16 / C>{}, Groups{});
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
