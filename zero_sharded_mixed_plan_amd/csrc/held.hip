// HIP kernels for gfx950 (CDNA4): matrices held in 8 bits, and the gated activation's
// gradient, which reads the two projections as they were or held in 8 bits.
//
// All stream: a lane takes 8 columns of a row, four lanes a block of 32.
#include <algorithm>

#include "held.h"

namespace zk {
namespace {

constexpr int kThreads8 = 256;

template <class T>
__global__ __launch_bounds__(kThreads8) void pack_kernel(const HoldLaunch a) {
  const u32 u = blockIdx.x * (u32)kThreads8 + threadIdx.x;
  const u32 row = quotient(u, a.groups), grp = u - row * a.groups.d;  // a quad lies in one row and block
  const u32 n = u < a.units && grp * 8 < a.cols ? min(a.cols - grp * 8, 8u) : 0;
  Raw8<T> r;
  load8<T>(a.x + (int64_t)row * a.ld_x + (int64_t)grp * 8 * T::bytes, a.x_end, n, r);
  float v[8];
  values8<T>(r, n, v);
  hold8(a.held, row, grp, v, n);
}

template <class T>
__global__ __launch_bounds__(kThreads8) void unpack_kernel(const HoldLaunch a) {
  const u32 u = blockIdx.x * (u32)kThreads8 + threadIdx.x;
  const u32 row = quotient(u, a.groups), grp = u - row * a.groups.d;
  const u32 n = u < a.units && grp * 8 < a.cols ? min(a.cols - grp * 8, 8u) : 0;
  if (n == 0) return;
  RawHeld r;
  load_held(a.held, row, grp, n, r);
  float v[8];
  held_values(r, n, v);
  store8<T>(a.x + (int64_t)row * a.ld_x + (int64_t)grp * 8 * T::bytes, v, n);
}

// a = g p u, dg = da u (p + g p q slope), du = da g p; see Gate.
template <class T, bool HELD, int ACT>
__global__ __launch_bounds__(kThreads8) void gated_grad_kernel(const GatedGradLaunch a) {
  const u32 i = blockIdx.x * (u32)kThreads8 + threadIdx.x;
  const u32 row = quotient(i, a.groups), grp = i - row * a.groups.d;
  const u32 n = i < a.units && grp * 8 < a.cols ? min(a.cols - grp * 8, 8u) : 0;
  if (n == 0) return;
  const int64_t col = (int64_t)grp * 8 * T::bytes;
  Raw8<T> rd;
  load8<T>(a.da + (int64_t)row * a.ld_da + col, a.da_end, n, rd);
  float d[8], g[8], u[8];
  if constexpr (HELD) {
    RawHeld qg, qu;
    load_held(a.hg, row, grp, n, qg);
    load_held(a.hu, row, grp, n, qu);
    held_values(qg, n, g);
    held_values(qu, n, u);
  } else {
    Raw8<T> rg, ru;
    load8<T>(a.g + (int64_t)row * a.ld_g + col, a.g_end, n, rg);
    load8<T>(a.u + (int64_t)row * a.ld_u + col, a.u_end, n, ru);
    values8<T>(rg, n, g);
    values8<T>(ru, n, u);
  }
  values8<T>(rd, n, d);
  float dg[8], du[8], act[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const Gate e = gate_of<T, ACT>(g[j]);
    const float v = g[j] * e.p;
    const float slope = __builtin_fmaf(v * e.q, e.slope, e.p);
    dg[j] = d[j] * u[j] * slope;
    du[j] = d[j] * v;
    act[j] = v * u[j];
  }
  store8<T>(a.dg + (int64_t)row * a.ld_dg + col, dg, n);
  store8<T>(a.du + (int64_t)row * a.ld_du + col, du, n);
  if (a.a) store8<T>(a.a + (int64_t)row * a.ld_a + col, act, n);
}

template <class F>
auto with_type(zero_dtype_t t, F&& f) {
  switch (t) {
    case ZERO_F32: return f(F32{});
    case ZERO_BF16: return f(BF16{});
    default: return f(F16{});
  }
}

u32 grid_of(u32 units) { return (u32)(((u64)units + kThreads8 - 1) / kThreads8); }

}  // namespace

int launch_pack(const HoldLaunch& a, zero_dtype_t t, void* stream) {
  return with_type(t, [&](auto x) {
    hipLaunchKernelGGL((pack_kernel<decltype(x)>), dim3(grid_of(a.units)), dim3(kThreads8), 0, (hipStream_t)stream, a);
    return launched("packing");
  });
}

int launch_unpack(const HoldLaunch& a, zero_dtype_t t, void* stream) {
  return with_type(t, [&](auto x) {
    hipLaunchKernelGGL((unpack_kernel<decltype(x)>), dim3(grid_of(a.units)), dim3(kThreads8), 0, (hipStream_t)stream, a);
    return launched("unpacking");
  });
}

int launch_gated_grad(const GatedGradLaunch& a, zero_dtype_t t, int32_t act, void* stream) {
  return with_type(t, [&](auto x) {
    using T = decltype(x);
    auto go = [&](auto held, auto kind) {
      hipLaunchKernelGGL((gated_grad_kernel<T, decltype(held)::value, decltype(kind)::value>), dim3(grid_of(a.units)),
                         dim3(kThreads8), 0, (hipStream_t)stream, a);
    };
    using Silu = std::integral_constant<int, kSilu>;
    using Gelu = std::integral_constant<int, kGelu>;
    if (a.hg.codes) act == kSilu ? go(std::true_type{}, Silu{}) : go(std::true_type{}, Gelu{});
    else act == kSilu ? go(std::false_type{}, Silu{}) : go(std::false_type{}, Gelu{});
    return launched("gated gradient");
  });
}

}  // namespace zk
